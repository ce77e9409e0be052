"""Residual + root-mean-square norm with bf16 and e4m3 outputs against the
definition in 64 bits.

Bounds: h is one fp32 addition (2^-24).  The sum of squares adds at most 32
terms in a thread, 5 and 32 across lanes and warps, 70 steps of 2^-24 relative
in all; its square root halves that, and mean, root, reciprocal and the two
products add 6 more: n is off by at most 2^-24 * 42 < 2^-18 relative before its
one rounding (half a step: bf16 2^-8; e4m3 2^-4, or half of the smallest step
2^-9 in units of the scale)."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -18


def data(T, d, seed, device=None, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d, generator=g) * gain).to(torch.bfloat16)
    r = (torch.randn(T, d, generator=g) * gain * 3).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
    return x, r, w


def near(got, want, half, extra=0.0):
    got = got.double()
    return ((got - want).abs() <= want.abs() * (half + ULP) + extra).all()


def check_q(q, s, n, group):
    T, d = n.shape
    g = group or d
    amax = n.view(T, -1, g).abs().amax(-1)
    want = torch.where(amax < 2.0 ** -100, 0.0, amax / 448)
    s = s.cpu().double().view(T, -1)
    assert ((s - want).abs() <= want * 2 * ULP).all()
    got = q.cpu().float().double().view(T, -1, g) * s[..., None]
    x = n.view(T, -1, g)
    tol = torch.maximum(x.abs() * 2.0 ** -4, 2.0 ** -10 * want[..., None]) + 4 * ULP * amax[..., None]
    assert ((got - x).abs() <= tol).all()


@pytest.mark.parametrize("T,d,group", [(1, 4096, 0), (3, 8, 0), (5, 64, 64), (33, 64, 16), (7, 2880, 32), (2, 4096, 128),
                                       (9, 120, 0), (130, 256, 256), (4, 264, 0), (3, 2168, 0), (2, 8192, 0), (2, 11008, 128),
                                       (3, 16384, 256), (2, 16392, 0), (2, 32768, 32), (1000, 512, 0), (17, 48, 16)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_against_the_definition(cuda_device, T, d, group, with_residual):
    x, r, w = data(T, d, T + d)
    h, n = R.norm(x, r if with_residual else None, w, 1e-5)
    dev = cuda_device
    xd, wd = x.to(dev), w.to(dev)
    rd = r.to(dev) if with_residual else None
    y, out = torch.empty_like(xd), torch.empty_like(xd)
    q = torch.empty(T, d, dtype=torch.float8_e4m3fn, device=dev)
    s = torch.empty((T, d // group) if group else (T,), device=dev)
    L.lora_rmsnorm(xd, wd, 1e-5, residual=rd, residual_out=out, y=y, q=q, q_scales=s)
    assert near(out.cpu(), h, R.U_BF16) and near(y.cpu(), n, R.U_BF16)
    check_q(q, s, n, group)
    # each output alone is the same
    y2, q2, s2 = torch.empty_like(y), torch.empty_like(q), torch.empty_like(s)
    L.lora_rmsnorm(xd, wd, 1e-5, residual=rd, y=y2)
    L.lora_rmsnorm(xd, wd, 1e-5, residual=rd, q=q2, q_scales=s2)
    assert torch.equal(y, y2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_in_place(cuda_device):
    x, r, w = data(37, 4096, 1)
    h, n = R.norm(x, r, w, 1e-6)
    xd, rd, wd = x.to(cuda_device), r.to(cuda_device), w.to(cuda_device)
    L.lora_rmsnorm(xd, wd, 1e-6, residual=rd, residual_out=rd, y=xd)
    assert near(rd.cpu(), h, R.U_BF16) and near(xd.cpu(), n, R.U_BF16)


def test_strided_rows(cuda_device):
    T, d = 11, 320
    x, r, w = data(T, d, 2)
    h, n = R.norm(x, r, w, 1e-5)
    wide = torch.full((T, 4 * d + 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    cols = [wide[:, i * (d + 8):i * (d + 8) + d] for i in range(4)]
    cols[0].copy_(x), cols[1].copy_(r)
    q = torch.zeros(T, d + 24, dtype=torch.uint8, device=cuda_device)
    s = torch.empty(T, 5, device=cuda_device)
    L.lora_rmsnorm(cols[0], w.to(cuda_device), 1e-5, residual=cols[1], residual_out=cols[2], y=cols[3],
                   q=q[:, :d].view(torch.float8_e4m3fn), q_scales=s)
    assert near(cols[2].cpu(), h, R.U_BF16) and near(cols[3].cpu(), n, R.U_BF16)
    check_q(q[:, :d].view(torch.float8_e4m3fn), s, n, 64)
    assert torch.equal(cols[0].cpu(), x) and torch.equal(cols[1].cpu(), r)
    assert (q[:, d:] == 0).all() and (wide[:, d:d + 8] == 7).all() and (wide[:, 4 * d + 24:] == 7).all()


def test_rows_of_zeros_small_and_large(cuda_device):
    d = 256
    x = torch.randn(5, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 55
    w = torch.ones(d, dtype=torch.bfloat16)
    for eps in (0.0, 1e-6):
        _, n = R.norm(x[1:], None, w, eps)
        y = torch.empty_like(x, device=cuda_device)
        q, s = torch.empty(5, d, dtype=torch.float8_e4m3fn, device=cuda_device), torch.empty(5, device=cuda_device)
        L.lora_rmsnorm(x.to(cuda_device), w.to(cuda_device), eps, y=y, q=q, q_scales=s)
        if eps:
            assert (y[0] == 0).all() and s[0] == 0 and (q[0].float() == 0).all()
        assert near(y[1:].cpu(), n, R.U_BF16)
        check_q(q[1:], s[1:], n, 0)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_value_that_is_not_finite_stays_with_its_row(cuda_device, bad):
    x, r, w = data(6, 512, 4)
    x[2, 77] = bad
    q, s = torch.empty(6, 512, dtype=torch.float8_e4m3fn, device=cuda_device), torch.empty(6, 16, device=cuda_device)
    y = torch.empty_like(x, device=cuda_device)
    L.lora_rmsnorm(x.to(cuda_device), w.to(cuda_device), 1e-5, residual=r.to(cuda_device), y=y, q=q, q_scales=s)
    ok = torch.tensor([0, 1, 3, 4, 5])
    assert torch.isfinite(y.cpu()[ok]).all() and torch.isfinite(s.cpu()[ok]).all()
    assert torch.isnan(y[2, 77]) and torch.isnan((q[2].float().view(16, 32) * s[2, :, None])[2]).all()


def test_refusals(cuda_device):
    x, r, w = (t.to(cuda_device) for t in data(4, 64, 5))
    y, q, s = torch.empty_like(x), torch.empty(4, 64, dtype=torch.float8_e4m3fn, device=cuda_device), torch.empty(4, device=cuda_device)

    def code(x=x, w=w, eps=1e-5, **more):
        with pytest.raises((L.LoraError, ValueError)) as e:
            L.lora_rmsnorm(x, w, eps, **more)
        return getattr(e.value, "code", None)

    n = L.lora_kernel_launches()
    assert code() == L.LORA_ERR_INVALID_ARG                                 # no output
    assert code(y=y, eps=-1.0) == L.LORA_ERR_INVALID_ARG and code(y=y, eps=float("nan")) == L.LORA_ERR_INVALID_ARG
    code(q=q), code(y=y.float()), code(y=y[:3]), code(w=w[:32], y=y), code(q=y, q_scales=s), code(y=y.cpu())
    code(q=q, q_scales=s[:2]), code(q=q, q_scales=torch.empty(4, 3, device=cuda_device))
    assert code(q=q, q_scales=torch.empty(4, 8, device=cuda_device)) == L.LORA_ERR_INVALID_ARG   # groups of 8
    assert code(x=x[:, :60].contiguous(), w=w[:60], y=y[:, :60]) == L.LORA_ERR_ALIGNMENT
    buf = torch.empty(4 * 64 + 64, dtype=torch.bfloat16, device=cuda_device)
    a, b = buf[:256].view(4, 64), buf[32:288].view(4, 64)
    assert code(x=a, y=b) == L.LORA_ERR_INVALID_ARG                         # a shifted overlap
    assert code(residual_out=y, y=y) == L.LORA_ERR_INVALID_ARG
    assert code(y=w.expand(1, 64), x=x[:1]) == L.LORA_ERR_INVALID_ARG
    assert L.lora_kernel_launches() == n
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=cuda_device)
    L.lora_rmsnorm(e, w, 1e-5, y=e.clone())
    assert L.lora_kernel_launches() == n


def test_stream_and_graph(cuda_device):
    x, r, w = (t.to(cuda_device) for t in data(64, 4096, 6))
    y, want = torch.empty_like(x), torch.empty_like(x)
    L.lora_rmsnorm(x, w, 1e-5, residual=r, y=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.lora_rmsnorm(x, w, 1e-5, residual=r, y=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w2 = w * 1.0  # made by another kernel right before: the launch may not read it early
        L.lora_rmsnorm(x, w2, 1e-5, residual=r, y=y)
    for _ in range(3):
        y.zero_(), w2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
