"""The cache's sticky status beside other streams: nothing that a call reports is lost, and reading it waits for
the named stream alone."""

import threading

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R
from test_gpu_kv import Cache

pytestmark = pytest.mark.gpu
BUSY = 600_000_000  # cycles: about 0.3 s


def bad_append(c, stream):
    b = c.b
    off, k, v = b.rows()
    L.lora_kv_append(c.kv, 0, k.to(c.device), v.to(c.device), c.table, c.bad, off.to(c.device), stream=stream)


@pytest.fixture
def batch():
    return R.Batch([20, 20], 2, 64, 16, seed=51)


def test_an_error_right_after_the_cache_is_made(cuda_device, batch):
    """The default stream is at work for a while; a call on another stream right after lora_kv_create fails."""
    side = torch.cuda.Stream()
    off, k, v = (t.to(cuda_device) for t in batch.rows())
    table, bad = batch.table.to(cuda_device), torch.tensor([33, 20], dtype=torch.int32, device=cuda_device)
    shape = (1, batch.n_pages, 16, 2, 64, 0)
    mem = torch.zeros(L.lora_kv_bytes_required(*shape), dtype=torch.uint8, device=cuda_device)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    kv = L.lora_kv_create(cuda_device.index, *shape, mem)
    try:
        L.lora_kv_append(kv, 0, k, v, table, bad, off, stream=side)
        torch.cuda.synchronize()
        assert L.lora_kv_get_error(kv, stream=side) == L.LORA_ERR_BAD_ID
        assert L.lora_kv_get_error(kv, stream=side) == L.LORA_OK
    finally:
        L.lora_kv_destroy(kv)


def test_reading_waits_for_its_stream_alone(cuda_device, batch):
    side = torch.cuda.Stream()
    with Cache(batch, "bf16", cuda_device) as c:
        c.bad = torch.tensor([33, 20], dtype=torch.int32, device=cuda_device)
        assert c.error() == L.LORA_OK  # (a kernel's first launch loads it, which may wait for the device)
        torch.cuda.synchronize()
        done = torch.cuda.Event()
        bad_append(c, side)
        side.synchronize()
        torch.cuda._sleep(BUSY)
        done.record()
        assert L.lora_kv_get_error(c.kv, stream=side) == L.LORA_ERR_BAD_ID
        assert not done.query()
        torch.cuda.synchronize()
        assert c.error() == L.LORA_OK


def test_readings_from_two_threads(cuda_device, batch):
    """Errors made on one stream while two threads read: each call has one row in error, which reports once, and is seen
    once; none is left at the end."""
    with Cache(batch, "int8", cuda_device) as c:
        c.append()
        bad = torch.tensor([33], dtype=torch.int32, device=cuda_device)
        assert c.error() == L.LORA_OK
        _, k, v = (t.to(cuda_device) for t in batch.rows())
        table = c.table[:1].contiguous()
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        seen, rounds = [0, 0], 200
        stop = threading.Event()

        def read(i):
            while not stop.is_set():
                e = L.lora_kv_get_error(c.kv, stream=streams[i])
                assert e in (L.LORA_OK, L.LORA_ERR_BAD_ID)
                seen[i] += e != L.LORA_OK

        threads = [threading.Thread(target=read, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        made = 0
        try:
            for _ in range(rounds):
                before = sum(seen)
                L.lora_kv_append(c.kv, 0, k[:1], v[:1], table, bad, stream=streams[2])
                made += 1
                streams[2].synchronize()
                for _ in range(100000):
                    if sum(seen) > before:
                        break
                    stop.wait(1e-4)
                assert sum(seen) == before + 1, "error %d was not reported once" % made
        finally:
            stop.set()
            for t in threads:
                t.join()
        assert c.error() == L.LORA_OK and sum(seen) == rounds
