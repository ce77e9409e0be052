"""Argument checks of the cache, attention and norm calls that come before any
device work, and the definitions the GPU tests compare with, without a GPU."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R


def test_sizes():
    # a token's key or value of a head: dim values, 8-bit ones with a 4-byte scale
    for kv_type, per in (("bf16", 2 * 128), ("e4m3", 128 + 4), ("int8", 128 + 4)):
        assert L.lora_kv_bytes_required(3, 10, 64, 8, 128, R.TYPES[kv_type]) == 3 * 10 * 64 * 8 * 2 * per
    for bad in ((0, 1, 16, 1, 16, 0), (1, 0, 16, 1, 16, 0), (1, 1, 15, 1, 16, 0), (1, 1, 48, 1, 16, 0),
                (1, 1, 2048, 1, 16, 0), (1, 1, 16, 0, 16, 0), (1, 1, 16, 1, 8, 0), (1, 1, 16, 1, 24, 0),
                (1, 1, 16, 1, 272, 0), (1, 1, 16, 1, 16, 3), (1, 1, 16, 1, 16, -1), (4097, 1, 16, 1, 16, 0),
                (4096, 2 ** 31 - 1, 1024, 1024, 256, 0)):
        assert L.lora_kv_bytes_required(*bad) == 0


def test_calls_without_a_cache_are_refused():
    lib, bad = L._lib, L.LORA_ERR_INVALID_ARG
    n = L.lora_kernel_launches()
    assert lib.lora_kv_append(None, 0, None, 0, None, 0, None, 0, None, None, 0, 0, None) == bad
    assert lib.lora_kv_gather(None, 0, None, 0, None, 0, None, 0, None, None, 0, 0, None) == bad
    assert lib.lora_attend(None, 0, None, 0, None, 0, None, None, 8, None, 0, None, 0, 1.0, 0, None, 0, None) == bad
    assert lib.lora_kv_destroy(None) == bad and lib.lora_kv_get_error(None, None, None) == bad
    assert lib.lora_attend_workspace_bytes(None, 8) == 0
    assert lib.lora_kv_create(None, 0, 1, 1, 16, 1, 16, 0, None, 0) == bad
    assert L.lora_kernel_launches() == n


A = 1 << 20  # addresses that no device call sees: every refusal comes first


def rms(x=A, ldx=64, r=2 * A, ldr=64, ro=3 * A, ldro=64, w=4 * A, eps=1e-5, y=5 * A, ldy=64, q=6 * A, ldq=64, s=7 * A,
        group=0, T=4, d=64):
    return L._lib.lora_rmsnorm(99, x, ldx, r, ldr, ro, ldro, w, eps, y, ldy, q, ldq, s, group, T, d, None)


def test_norm_refusals():
    inv, al = L.LORA_ERR_INVALID_ARG, L.LORA_ERR_ALIGNMENT
    refused = dict(
        inv=[dict(x=None), dict(w=None), dict(y=None, q=None), dict(s=None), dict(T=-1), dict(T=(1 << 20) + 1),
             dict(d=0), dict(d=32776, ldx=32776), dict(ldx=56), dict(ldr=56), dict(ldro=56), dict(ldy=56), dict(ldq=56),
             dict(eps=-1.0), dict(group=8), dict(group=48), dict(group=512), dict(group=128), dict(group=-16),
             dict(y=A + 64), dict(ro=A + 128), dict(y=2 * A + 8 * 2), dict(y=3 * A), dict(q=5 * A + 64), dict(y=4 * A),
             dict(s=5 * A), dict(s=A + 16), dict(y=A, ldy=72), dict(q=A)],
        al=[dict(x=A + 8), dict(r=2 * A + 2), dict(ro=3 * A + 8), dict(w=4 * A + 4), dict(y=5 * A + 8), dict(q=6 * A + 8),
            dict(s=7 * A + 2), dict(ldx=68), dict(ldq=68), dict(d=60)])
    for want, cases in ((inv, refused["inv"]), (al, refused["al"])):
        for c in cases:
            assert rms(**c) == want, c
    assert rms(T=0) == L.LORA_OK


def test_binding_refuses_what_the_pointers_cannot_show():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(Exception):  # no device tensor
        L.lora_rmsnorm(x, w, 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError):
        L.lora_rmsnorm(x.float(), w, 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError):
        L.lora_rmsnorm(x, w, 1e-5, y=torch.empty_like(x)[:3])


def test_the_definition_against_torch_conversion():
    x = torch.linspace(-448, 448, 4001).double()
    assert torch.equal(R.round_e4m3(x).float(), x.float().to(torch.float8_e4m3fn).float())
    small = torch.linspace(-2.0 ** -6, 2.0 ** -6, 1001).double()
    assert torch.equal(R.round_e4m3(small).float(), small.float().to(torch.float8_e4m3fn).float())


def test_the_definition_of_attention_by_hand():
    # two tokens, equal keys: the mean of the values; a sink of the same score takes a third
    q, k = torch.ones(1, 16).bfloat16(), torch.ones(2, 1, 16).bfloat16()
    v = torch.stack([torch.zeros(1, 16), torch.full((1, 16), 3.0)]).bfloat16()
    out, lse, _, _ = R.attend(q, k, v, "bf16", 0.25)
    assert torch.allclose(out, torch.full((1, 16), 1.5).double()) and abs(lse.item() - (4 + 0.6931471805599453)) < 1e-12
    out, _, _, _ = R.attend(q, k, v, "bf16", 0.25, sinks=torch.tensor([4.0]))
    assert torch.allclose(out, torch.ones(1, 16).double())
    out, _, _, _ = R.attend(q, k, v, "bf16", 0.25, window=1)
    assert torch.allclose(out, torch.full((1, 16), 3.0).double())
