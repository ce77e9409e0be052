"""Rows of which no token is left, or none has any weight: zeros and the sink alone, as for a length of 0."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R
from test_gpu_attend import attend, check, queries
from test_gpu_kv import Cache

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (16, 1, 256), (20, 2, 48)])
def test_no_page_of_a_sequence_is_in_the_cache(cuda_device, kv_type, heads, kv_heads, dim):
    """A short sequence (one warp's) and a long one (cut over many blocks) whose pages are all outside, between others."""
    b = R.Batch([40, 1, 100, 30000, 77], kv_heads, dim, 16, seed=41)
    q = queries(b, heads, 41)
    sinks = torch.linspace(-3, 3, heads)
    sinks[1] = -INF
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        assert c.error() == L.LORA_OK
        good, good_lse = attend(c, q)
        c.table[1] = -1
        c.table[3] = b.n_pages
        out, lse = attend(c, q)
        assert c.error() == L.LORA_ERR_BAD_ID
        keep = [0, 2, 4]
        assert (out[[1, 3]] == 0).all() and (lse[[1, 3]] == -INF).all()
        assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], good_lse[keep])
        out, lse = attend(c, q, sinks=sinks)
        assert c.error() == L.LORA_ERR_BAD_ID
        assert (out[[1, 3]] == 0).all()
        # the sink passes through base 2 and back: two products' roundings
        fin = torch.isfinite(sinks)
        assert ((lse[[1, 3]][:, fin] - sinks[fin]).abs() <= 3 * 2.0 ** -24 * sinks[fin].abs()).all()
        assert (lse[[1, 3]][:, ~fin] == -INF).all()


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_the_window_is_on_no_page(cuda_device, kv_type):
    b = R.Batch([100, 64], 2, 64, 16, seed=42)
    q = queries(b, 8, 42)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        c.table[0, 5:] = -7  # tokens 80 to 99
        out, lse = attend(c, q, window=20)
        assert c.error() == L.LORA_ERR_BAD_ID
        assert (out[0] == 0).all() and (lse[0] == -INF).all()
        assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all() and (out[1] != 0).any()
        c.table.copy_(b.table)
        check(c, kv_type, q, *attend(c, q, window=20), window=20)


def test_all_scores_are_minus_infinity(cuda_device):
    """Keys of -inf against positive q: no weight, so zeros; one finite key among them takes all of it."""
    b = R.Batch([50, 3000], 1, 64, 16, seed=43)
    q = torch.ones(2, 4 * 64, dtype=torch.bfloat16)
    for k in b.k:
        k.fill_(-INF)
    with Cache(b, "bf16", cuda_device) as c:
        c.append()
        out, lse = attend(c, q)
        assert (out == 0).all() and (lse == -INF).all()
        out, lse = attend(c, q, sinks=torch.tensor([0.0, -INF, 2.0, 1.0]))
        assert (out == 0).all() and (lse[:, 1] == -INF).all() and (lse[:, 0] == 0).all()
    for k in b.k:
        k[33] = 0
    with Cache(b, "bf16", cuda_device) as c:
        c.append()
        out, lse = attend(c, q)
        for i in range(2):
            # (the base-2 logarithm is good to 2^-22; ln 2 times it and the reference, at most 4, add two roundings of
            # 2^-24 * 4: under 2^-20 in all)
            assert torch.equal(out[i].view(4, 64), b.v[i][33].expand(4, 64)) and (lse[i].abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_scores_that_are_nan_stay_so(cuda_device, kv_type):
    b = R.Batch([50, 50], 1, 64, 16, seed=44)
    q = queries(b, 4, 44)
    q[0, 64] = float("nan")  # head 1
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        out, lse = attend(c, q)
        out = out.view(2, 4, 64)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
        assert torch.isfinite(out[1]).all() and torch.isfinite(out[0, [0, 2, 3]]).all() and torch.isfinite(lse[0, [0, 2, 3]]).all()
