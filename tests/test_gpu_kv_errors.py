"""What calls in error write: nothing of a sequence in error, the others whole, and rows that offsets in disorder leave
in doubt either where some sequence wants them or nowhere."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R
from test_gpu_kv import Cache

pytestmark = pytest.mark.gpu
LENS = [20, 20, 20, 20]


def new_rows(b, seed):
    """Other values for the same tokens."""
    n = R.Batch(b.lens, b.kv_heads, b.dim, b.page, seed=seed)
    return n, [t for t in n.rows()]


def held(c, kv_type):
    """Every token as the cache has it: K and V [tokens, width]."""
    k, v = c.gather()
    assert c.error() == L.LORA_OK
    return k, v


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("lens,wrong", [([20, 33, 20, 20], 1), ([20, 20, -2, 20], 2), ([20, 20, 20, 19], 3),
                                        ([1 << 30, 20, 20, 20], 0), ([20, -(1 << 31), 20, 20], 1), ([0, 20, 20, 20], 0)])
def test_no_row_of_a_sequence_in_error_is_written(cuda_device, kv_type, lens, wrong):
    b = R.Batch(LENS, 2, 64, 16, seed=61)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        old = held(c, kv_type)
        before = c.mem.clone()
        other, (off, k, v) = new_rows(b, 62)
        L.lora_kv_append(c.kv, 0, k.to(cuda_device), v.to(cuda_device), c.table,
                         torch.tensor(lens, dtype=torch.int32, device=cuda_device), off.to(cuda_device))
        assert c.error() == L.LORA_ERR_BAD_ID
        got = held(c, kv_type)
        for g, o, x in zip(got, old, (k, v)):
            want = R.read_back(x.view(-1, 2, 64), kv_type).view(x.shape).clone()
            want[20 * wrong:20 * wrong + 20] = o[20 * wrong:20 * wrong + 20]
            assert torch.equal(g, want)
        # what holds no token is left as well: with the right rows back, memory is as it was
        c.append()
        assert c.error() == L.LORA_OK and torch.equal(before, c.mem)


LOWEST, HIGHEST = -(1 << 31), (1 << 31) - 1


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("off,whole", [
    ([0, 20, 40, 60, 81], [0, 1, 2]), ([-1, 20, 40, 60, 80], [1, 2, 3]), ([0, 30, 20, 60, 80], []),
    ([20, 40, 60, 80, 0], []), ([80, 60, 40, 20, 0], []), ([5, 5, 5, 5, 4], []),
    ([LOWEST, HIGHEST, HIGHEST, HIGHEST, HIGHEST], []), ([LOWEST, LOWEST, -1, HIGHEST, HIGHEST], []),
    ([HIGHEST, 20, 40, 60, LOWEST], []), ([0, 20, HIGHEST, 60, 80], [])])
def test_offsets_in_disorder(cuda_device, kv_type, off, whole):
    """Each token is as before, or a row that its sequence's offsets give it; sequences beside an end out of range are
    whole."""
    b = R.Batch(LENS, 2, 64, 16, seed=63)
    T = 80
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        old = held(c, kv_type)
        before = c.mem.clone()
        other, (_, k, v) = new_rows(b, 64)
        o = torch.tensor(off, dtype=torch.int32, device=cuda_device)
        L.lora_kv_append(c.kv, 0, k.to(cuda_device), v.to(cuda_device), c.table, c.lens, o)
        assert c.error() == L.LORA_ERR_BAD_ID
        got = held(c, kv_type)
        for g, was, x in zip(got, old, (k, v)):
            new = R.read_back(x.view(-1, 2, 64), kv_type).view(x.shape)
            for s in range(4):
                own = off[s + 1] - off[s]
                for pos in range(20):
                    t = off[s + 1] - (20 - pos)  # the row that would be this token
                    mine = own <= 20 and max(off[s], 0) <= t < min(off[s + 1], T)
                    at = 20 * s + pos
                    ok = [was[at]] if s not in whole else []
                    if mine:
                        ok.append(new[t])
                    assert any(torch.equal(g[at], y) for y in ok), (s, pos)
        # the read-back with the same offsets skips what is in doubt
        ko = torch.full_like(k, 7.0, device=cuda_device)
        vo = torch.full_like(v, 7.0, device=cuda_device)
        L.lora_kv_gather(c.kv, 0, ko, vo, c.table, c.lens, o)
        assert c.error() == L.LORA_ERR_BAD_ID
        for out, g in ((ko.cpu(), got[0]), (vo.cpu(), got[1])):
            for t in range(T):
                ok = [torch.full((128,), 7.0, dtype=torch.bfloat16)]
                for s in range(4):
                    if off[s] <= t < off[s + 1] and off[s + 1] - off[s] <= 20:
                        ok.append(g[20 * s + 20 - (off[s + 1] - t)])
                        if s in whole:
                            ok = ok[1:]
                assert any(torch.equal(out[t], y) for y in ok), t
        c.append()
        assert c.error() == L.LORA_OK and torch.equal(before, c.mem)
