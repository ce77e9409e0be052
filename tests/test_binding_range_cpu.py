"""Sizes and indices past a C int: the binding refuses them, ctypes would cut them to 32 bits unseen.  No GPU:
tensors without memory, and the library's calls replaced by ones that note what arrives."""

import ctypes

import pytest
import torch

import adapter_deltas_b200 as L

BIG = 1 << 32
BF16 = torch.bfloat16


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.fixture
def calls(monkeypatch):
    """What the C calls would see of their int arguments."""
    seen = []
    for name in ("lora_kv_append", "lora_kv_gather", "lora_attend", "lora_rmsnorm", "lora_kv_create"):
        types = getattr(L._lib, name).argtypes

        def note(*args, types=types, name=name):
            assert len(args) == len(types)
            seen.append((name, [ctypes.c_int(a).value for a, t in zip(args, types) if t is ctypes.c_int]))
            return L.LORA_OK

        monkeypatch.setattr(L._lib, name, note)
    return seen


def cache():
    return L.KvHandle(1, -1, None, 2, 8, 16, 2, 64, 0)


def rows(n=2, T=None, pages=4):
    return (meta(n, pages, dtype=torch.int32), meta(n, dtype=torch.int32),
            None if T is None else meta(n + 1, dtype=torch.int32))


def refused(call):
    with pytest.raises(L.LoraError) as e:
        call()
    return e.value.code == L.LORA_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", ["lora_kv_append", "lora_kv_gather"])
def test_cache_calls(calls, fn):
    call = getattr(L, fn)
    table, lens, off = rows(T=3)
    k = meta(3, 128)
    call(cache(), 1, k, k, table, lens, off, stream=0)
    assert calls == [(fn, [1, 128, 128, 4, 2, 3])]
    for layer in (BIG, BIG + 1, -1, -BIG, 1 << 31):
        assert refused(lambda: call(cache(), layer, k, k, table, lens, off, stream=0))
    far = torch.empty_strided((3, 128), (BIG + 128, 1), dtype=BF16, device="meta")
    assert refused(lambda: call(cache(), 0, far, k, table, lens, off, stream=0))
    assert refused(lambda: call(cache(), 0, k, far, table, lens, off, stream=0))
    many = meta(BIG + 3, 128)
    assert refused(lambda: call(cache(), 0, many, many, table, lens, off, stream=0))
    table, lens, _ = rows(n=BIG + 3)
    assert refused(lambda: call(cache(), 0, k, k, table, lens, None, stream=0))
    assert len(calls) == 1


def test_attention(calls):
    table, lens, _ = rows()
    q, ws = meta(2, 256), meta(1024, dtype=torch.uint8)
    L.lora_attend(cache(), 0, q, q, table, lens, ws, stream=0)
    assert calls.pop() == ("lora_attend", [0, 256, 256, 4, 4, 2, 0])
    for window, arrives in ((7, 7), (1 << 30, 1 << 30), (BIG + 5, 1 << 30), (1 << 80, 1 << 30)):
        L.lora_attend(cache(), 0, q, q, table, lens, ws, window=window, stream=0)
        assert calls.pop()[1][-1] == arrives  # no sequence is longer than 2^30
    for window in (-1, -BIG, -BIG + 5):
        assert refused(lambda: L.lora_attend(cache(), 0, q, q, table, lens, ws, window=window, stream=0))
    for layer in (BIG, -BIG):
        assert refused(lambda: L.lora_attend(cache(), layer, q, q, table, lens, ws, stream=0))
    far = torch.empty_strided((2, 256), (BIG + 256, 1), dtype=BF16, device="meta")
    assert refused(lambda: L.lora_attend(cache(), 0, far, q, table, lens, ws, stream=0))
    assert refused(lambda: L.lora_attend(cache(), 0, q, far, table, lens, ws, stream=0))
    many = meta(2, 64 * (BIG + 4))
    assert refused(lambda: L.lora_attend(cache(), 0, many, many, table, lens, ws, stream=0))
    assert not calls


def test_norm(calls):
    w, y = meta(64), meta(4, 64)
    L.lora_rmsnorm(y, w, 1e-5, y=y, stream=0)
    assert calls.pop()[1][-2:] == [4, 64]
    many = meta(BIG + 4, 64)
    assert refused(lambda: L.lora_rmsnorm(many, w, 1e-5, y=many, stream=0))
    wide = meta(2, BIG + 64)
    assert refused(lambda: L.lora_rmsnorm(wide, meta(BIG + 64), 1e-5, y=wide, stream=0))
    far = torch.empty_strided((4, 64), (BIG + 64, 1), dtype=BF16, device="meta")
    for more in (dict(x=far), dict(residual=far), dict(residual_out=far), dict(y=far)):
        args = dict(dict(x=y, weight=w, eps=1e-5, y=y, stream=0), **more)
        assert refused(lambda: L.lora_rmsnorm(**args))
    assert not calls


def test_sizes_and_creation(calls):
    for i in range(6):
        shape = [1, 4, 16, 2, 64, 0]
        shape[i] += BIG
        assert L.lora_kv_bytes_required(*shape) == 0
        assert refused(lambda: L.lora_kv_create(-1, *shape, meta(1 << 20, dtype=torch.uint8)))
        shape[i] -= 2 * BIG
        assert L.lora_kv_bytes_required(*shape) == 0
    assert not calls
