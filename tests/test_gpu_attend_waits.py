"""The attention's bounded waits: what a warp does when they run out."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R
from test_gpu_attend import attend, queries
from test_gpu_kv import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lane", [0, 17, 31])
@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_a_wait_that_runs_out_for_one_lane_ends_its_warp(cuda_device, kv_type, lane):
    """All data arrive, but one lane's clock says that they came too late: the warp gives up as one, with its copies
    landed, and rows are left alone or right."""
    b = R.Batch([150000, 33, -1, 5, 250000, 0] + [40] * 300, 2, 64, 16, seed=20)
    q = queries(b, 8, 20)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        ws = torch.full((L.lora_attend_workspace_bytes(c.kv, 8),), 255, dtype=torch.uint8, device=cuda_device)
        want, _ = attend(c, q, ws=ws, scale=1.0)
        assert c.error() == L.LORA_OK
        qd = q.to(cuda_device)
        for _ in range(3):
            out = torch.full_like(qd, 7.0)
            L.lora_set_wait_limit_ns(20_000_000)
            try:
                L.lora_selftest_late_lane_attend(c.kv, 0, qd, out, c.table, c.lens, ws, lane)
                torch.cuda.synchronize()
            finally:
                L.lora_set_wait_limit_ns(0)
            assert c.error() == L.LORA_ERR_TIMEOUT and c.error() == L.LORA_OK
            heads = out.cpu().view(-1, 8, 64)
            left = (heads == 7.0).all(-1)
            assert left[0].all() and left[4].all()  # cut over many warps, most of which have a third step
            assert not left[6:].all() and torch.equal(heads[~left], want.view(-1, 8, 64)[~left])
            got, _ = attend(c, q, ws=ws, scale=1.0)
            assert torch.equal(got, want) and c.error() == L.LORA_OK


def test_late_lane_refusals(cuda_device):
    b = R.Batch([20], 2, 64, 16, seed=21)
    q = queries(b, 4, 21).to(cuda_device)
    with Cache(b, "bf16", cuda_device) as c:
        ws = torch.empty(L.lora_attend_workspace_bytes(c.kv, 4), dtype=torch.uint8, device=cuda_device)
        n = L.lora_kernel_launches()
        for lane in (-1, 32):
            with pytest.raises(L.LoraError) as e:
                L.lora_selftest_late_lane_attend(c.kv, 0, q, torch.empty_like(q), c.table, c.lens, ws, lane)
            assert e.value.code == L.LORA_ERR_INVALID_ARG
        assert L.lora_kernel_launches() == n


@pytest.mark.parametrize("kv_type,dim", [("bf16", 16), ("e4m3", 16), ("int8", 64), ("bf16", 256)])
def test_giving_up_takes_one_limit(cuda_device, kv_type, dim):
    """Nothing is fetched, so nothing is in flight: a launch that gives up ends after one limit, however many stages a
    warp's ring has (8 of 16 dims)."""
    b = R.Batch([3000, 500], 2, dim, 16, seed=22)
    q = queries(b, 8, 22)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        ws = torch.full((L.lora_attend_workspace_bytes(c.kv, 8),), 255, dtype=torch.uint8, device=cuda_device)
        want, _ = attend(c, q, ws=ws)
        qd = q.to(cuda_device)
        out = torch.full_like(qd, 7.0)
        limit = 0.1  # counted in cycles of a 2 GHz clock: up to 2 GHz / the SM's clock times as long
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        L.lora_set_wait_limit_ns(int(limit * 1e9))
        try:
            start.record()
            L.lora_selftest_stalled_attend(c.kv, 0, qd, out, c.table, c.lens, ws)
            end.record()
            torch.cuda.synchronize()
        finally:
            L.lora_set_wait_limit_ns(0)
        assert 0.9 * limit <= start.elapsed_time(end) * 1e-3 <= 2.5 * limit
        assert c.error() == L.LORA_ERR_TIMEOUT and (out == 7.0).all()
        got, _ = attend(c, q, ws=ws)
        assert torch.equal(got, want) and c.error() == L.LORA_OK
