"""The norm over bf16's whole range: rows whose squares pass fp32's range, and rows
too small for their squares' bits where eps is next to nothing.  The bounds are
test_gpu_norm's; squares are taken in units of 2^80 then, which are exact, and
1 / rms of the largest rows (down to 2^-128) has 2^-22 of itself, inside the 2^-18
there.  Results below bf16's normal range are off by half of its smallest step, 2^-134."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R
from test_gpu_norm import check_q, near

pytestmark = pytest.mark.gpu


def run(x, w, eps, device, residual=None, group=0):
    T, d = x.shape
    xd, wd = x.to(device), w.to(device)
    y, out = torch.empty_like(xd), torch.empty_like(xd)
    q = torch.empty(T, d, dtype=torch.float8_e4m3fn, device=device)
    s = torch.empty((T, d // group) if group else (T,), device=device)
    L.lora_rmsnorm(xd, wd, eps, residual=None if residual is None else residual.to(device), residual_out=out, y=y, q=q,
                   q_scales=s)
    return out, y, q, s


EXPONENTS = [0, 50, 58, 62, 64, 70, 100, 124, -20, -50, -55, -64, -70, -100, -120, -128]


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-12, 1e-5])
@pytest.mark.parametrize("d", [64, 256, 512, 2880, 4096, 16384])
@pytest.mark.parametrize("many", [False, True])
def test_rows_of_every_magnitude(cuda_device, d, eps, many):
    """Rows of all magnitudes side by side (where d is small in one warp, between ordinary ones)."""
    g = torch.Generator().manual_seed(d)
    T = 700 if many and d <= 4096 else 33  # (over 4 rows an SM another variant takes them)
    x = torch.randn(T, d, generator=g).double()
    e = torch.tensor([EXPONENTS[i % len(EXPONENTS)] for i in range(T)])
    x = (x * torch.exp2(e.double())[:, None]).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
    h, n = R.norm(x, None, w, eps)
    if eps == 0:
        assert (n.square().mean(-1) > 0.5).all()  # every row is a row of ordinary numbers
    out, y, q, s = run(x, w, eps, cuda_device, group=64)
    assert torch.equal(out.cpu(), x)
    assert near(y.cpu(), n, R.U_BF16, extra=2.0 ** -134)
    amax = n.abs().amax(-1)
    held = n.view(T, -1, 64).abs().amax(-1).amin(-1) >= 2.0 ** -100  # (groups below that are held as zeros)
    check_q(q[held.to(cuda_device)], s[held.to(cuda_device)], n[held], 64)
    none = (amax < 2.0 ** -100).to(cuda_device)
    assert (s[none] == 0).all() and (q[none].float() == 0).all()


@pytest.mark.parametrize("d", [128, 1024, 8192])
def test_rows_of_mixed_magnitudes(cuda_device, d):
    """One large value among small ones, with and without a residual that cancels it."""
    g = torch.Generator().manual_seed(d + 1)
    x = torch.randn(12, d, generator=g)
    for i, e in enumerate((60, 64, 80, 126, -60, -126)):
        x[i, i + 3] *= 2.0 ** e
        x[6 + i] *= 2.0 ** -40
        x[6 + i, 5] = 2.0 ** (e / 2)
    x = x.to(torch.bfloat16)
    r = torch.randn(12, d, generator=g).to(torch.bfloat16)
    r[0, 3], r[2, 5] = -x[0, 3], -x[2, 5]
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
    for residual in (None, r):
        for eps in (0.0, 1e-6):
            h, n = R.norm(x, residual, w, eps)
            out, y, q, s = run(x, w, eps, cuda_device, residual=residual)
            assert near(out.cpu(), h, R.U_BF16, extra=2.0 ** -134) and near(y.cpu(), n, R.U_BF16, extra=2.0 ** -134)


def test_infinite_and_nan_rows_between(cuda_device):
    x = torch.randn(8, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    x[1, 3], x[3, 4] = float("inf"), float("nan")
    x[5] *= 2.0 ** 90
    w = torch.ones(64, dtype=torch.bfloat16)
    _, y, _, _ = run(x, w, 0.0, cuda_device)
    ok = [0, 2, 4, 5, 6, 7]
    _, n = R.norm(x[ok], None, w, 0.0)
    assert near(y.cpu()[ok], n, R.U_BF16)
    assert torch.isnan(y[1, 3]) and torch.isnan(y[3]).all()
