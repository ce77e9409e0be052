"""Sinks over fp32's whole range: as a mask (the lowest value, minus infinity) and as what takes all the weight."""

import pytest
import torch

import kv_reference as R
from test_gpu_attend import attend, check, queries
from test_gpu_kv import Cache

pytestmark = pytest.mark.gpu
TOP = torch.finfo(torch.float32).max
INF = float("inf")


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("lens", [[1, 300, 0, 40], [20000, 0, 33]])
def test_sinks_at_the_ends_of_the_range(cuda_device, kv_type, lens):
    b = R.Batch(lens, 2, 64, 16, seed=71)
    q = queries(b, 8, 71)
    sinks = torch.tensor([-TOP, TOP, -INF, -2.4e38, 2.4e38, 3e38, -3e38, 0.5])
    large = torch.tensor([1, 4, 5])
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        out, lse = attend(c, q, sinks=sinks)
        # (the definition in 64 bits; the log-sum-exp under a sink of 1e38 is that sink)
        check(c, kv_type, q, out, lse, sinks=sinks)
        bare, bare_lse = attend(c, q)
        small = torch.tensor([0, 2, 3, 6])
        heads = lambda t: t.view(len(lens), 8, 64)  # noqa: E731
        assert torch.equal(heads(out)[:, small], heads(bare)[:, small])
        assert (heads(out)[:, large] == 0).all() and torch.equal(lse[:, large], sinks[large].expand(len(lens), 3))
        full = [i for i, n in enumerate(lens) if n]
        assert torch.equal(lse[full][:, small], bare_lse[full][:, small])
        # no token left: the sink alone, as it was given
        c.table.fill_(-1)
        out, lse = attend(c, q, sinks=sinks)
        c.error()
        assert (out == 0).all() and torch.equal(lse, sinks.expand(len(lens), 8))


def test_sinks_that_are_infinite_or_nan(cuda_device):
    b = R.Batch([30], 1, 64, 16, seed=72)
    q = queries(b, 3, 72)
    with Cache(b, "bf16", cuda_device) as c:
        c.append()
        out, lse = attend(c, q, sinks=torch.tensor([INF, float("nan"), 0.0]))
        out = out.view(3, 64)
        assert torch.isnan(out[:2]).all() and torch.isnan(lse[0, 1]) and torch.isfinite(out[2]).all()
