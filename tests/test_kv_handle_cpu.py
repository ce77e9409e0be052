"""The cache's handle after it is gone, without a GPU: the library's calls are replaced by ones that note their handle."""

import pytest

import adapter_deltas_b200 as L


@pytest.mark.parametrize("code", [L.LORA_OK, L.LORA_ERR_CUDA])
def test_a_handle_is_passed_to_destroy_once(monkeypatch, code):
    """lora_kv_destroy frees the handle whatever it reports: a second call must not pass it again."""
    seen = []
    monkeypatch.setattr(L._lib, "lora_kv_destroy", lambda kv: seen.append(getattr(kv, "ptr", kv)) or code)
    kv = L.KvHandle(4096, 0, None, 1, 4, 16, 2, 64, 0)
    if code == L.LORA_OK:
        L.lora_kv_destroy(kv)
    else:
        with pytest.raises(L.LoraError):
            L.lora_kv_destroy(kv)
    L.lora_kv_destroy(kv)
    assert seen == [4096] and not kv.ptr
