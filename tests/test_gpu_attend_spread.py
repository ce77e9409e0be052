"""Attention over caches whose rows differ widely in magnitude.

Every row of an 8-bit cache has its own scale, so rows of 2^-100 and of 2^100 may
lie side by side, and how large a row is says nothing about how much weight its
token gets.  The results are held to bounds that follow the terms which count:

  - a score is off by err_s as kv_reference.attend derives it; a weight by twice
    that relatively, plus 2^-15 for the exponential and the running rescale, plus
    len * 2^-23 for the sums;
  - 8-bit caches round a weight times its row's scale to fp16, 2^-11 relative; its
    exponent is a sum of the score s in base 2 and the scale's logarithm, two
    roundings of up to 2^-24 (|s| + 128) each and 2^-22 * 128 of the logarithm, times
    ln 2;
  - such a product is held in units in which the largest of them is at least 2^11,
    so that fp16's half smallest step 2^-25 is at most 2^-36 of the largest, for each
    of len tokens, times the largest code;
  - the result is rounded to bf16 once (2^-8; 2^-134 below its normal range).
"""

import math

import pytest
import torch

import kv_reference as R
from test_gpu_attend import attend, queries
from test_gpu_kv import Cache

pytestmark = pytest.mark.gpu


def expected(q, k, v, kv_type, scale, window=0):
    """One sequence's result [heads, dim] and what it may be off by."""
    heads, dim = q.shape
    if window and len(k) > window:
        k, v = k[-window:], v[-window:]
    n, kv_heads = len(k), k.shape[1]
    kx, (code, u) = R.values(k, kv_type).transpose(0, 1), R.held(v, kv_type)
    vx = (code * u[..., None]).transpose(0, 1)
    qx = q.double().view(kv_heads, -1, dim)
    s = scale * qx @ kx.transpose(1, 2)
    mag = (scale * qx.abs() @ kx.abs().transpose(1, 2)).amax(-1)
    p = torch.softmax(s, -1)
    out, spread = p @ vx, p @ vx.abs()
    rel = 2 * mag * (dim + 4) * 2.0 ** -23 + 2.0 ** -15 + n * 2.0 ** -23
    floor = torch.zeros_like(rel)
    if kv_type != "bf16":
        s2 = (mag * math.log2(math.e) + 128)
        rel = rel + 2.0 ** -11 + math.log(2) * (2 * 2.0 ** -24 * s2 + 2.0 ** -22 * 128)
        top = (p * u.transpose(0, 1)[:, None]).amax(-1)
        floor = n * 2.0 ** -36 * R.QMAX[kv_type] * top
    tol = R.U_BF16 * out.abs() + (rel[..., None] * spread + floor[..., None]) * (1 + R.U_BF16) + 2.0 ** -134
    return out.reshape(heads, dim), tol.reshape(heads, dim)


def hold(b, kv_type, q, out, window=0):
    for i, n in enumerate(b.lens):
        want, tol = expected(q[i].view(-1, b.dim), b.k[i], b.v[i], kv_type, b.dim ** -0.5, window)
        got = out[i].view(-1, b.dim).double()
        off = ((got - want).abs() / tol).max() if torch.isfinite(got).all() else float("nan")
        assert off <= 1, "sequence %d of length %d: %s of what it may be off" % (i, n, off)


def gains(n, way):
    """Powers of two (nearly) that the V rows of n tokens are multiplied by."""
    x = torch.linspace(0, 1, n) if n > 1 else torch.zeros(1)
    if way == "grow":
        return torch.exp2(60 * x - 30)
    if way == "shrink":
        return torch.exp2(30 - 60 * x)
    g = torch.Generator().manual_seed(n)
    steps = torch.tensor([1.0, 5.0, 100.0, 2.0 ** 20, 2.0 ** -20, 2.0 ** -40])
    if way == "jump":
        return steps[torch.randint(len(steps), (n,), generator=g)]
    return steps[torch.randint(len(steps), (n // 50 + 1,), generator=g)].repeat_interleave(50)[:n]  # "levels"


LENS = [[512, 1, 17, 300, 64], [30000, 7]]


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("way", ["grow", "shrink", "jump", "levels"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (4, 4, 128), (16, 1, 256), (20, 2, 48)])
def test_values_that_grow_shrink_and_jump(cuda_device, kv_type, way, lens, heads, kv_heads, dim):
    b = R.Batch(lens, kv_heads, dim, 32, seed=31)
    for v in b.v:
        v.copy_((v.float() * gains(len(v), way)[:, None, None]).to(torch.bfloat16))
    q = queries(b, heads, 31)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        hold(b, kv_type, q, attend(c, q)[0])
        hold(b, kv_type, q, attend(c, q, window=100)[0], window=100)
        assert c.error() == 0


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("spread", [8, 20, 26, 30, 34, 60, 100])
@pytest.mark.parametrize("lens,at", [([512, 90], 3), ([512, 90], 70), ([30000, 500], 5), ([30000, 500], 499)])
def test_a_large_value_without_weight(cuda_device, kv_type, spread, lens, at):
    """One token has V 2^spread times the others' and a score far below theirs: nothing of it is to be seen."""
    b = R.Batch(lens, 2, 64, 16, seed=32)
    q = queries(b, 8, 32)
    g = q.view(len(lens), 2, 4, 64)
    g.copy_(g[:, :, :1] + 0.1 * g)  # the heads of a key head look the same way
    for i in range(len(lens)):
        mean = g[i].float().mean(1)  # [kv_heads, dim]
        b.k[i][at] = (-mean / mean.square().sum(-1, keepdim=True) * 200 * 8).to(torch.bfloat16)  # score about -200
        b.v[i][at] *= 2.0 ** spread
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        hold(b, kv_type, q, attend(c, q)[0])


@pytest.mark.parametrize("kv_type", ["e4m3", "int8"])
def test_small_and_no_values(cuda_device, kv_type):
    """Rows of zeros hold the largest weights, and what is left is near the end of the types' ranges."""
    b = R.Batch([400, 33, 20000], 2, 64, 16, seed=33)
    for v in b.v:
        v[::2] = 0
        v[1::2] = (v[1::2].float() * 2.0 ** -96).to(torch.bfloat16)
    q = queries(b, 8, 33, gain=4.0)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        hold(b, kv_type, q, attend(c, q)[0])
    for v in b.v:
        v.zero_()
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        out, lse = attend(c, q)
        assert (out == 0).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("spread", [5, 10, 14, 17, 18, 20, 24, 30, 60])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (4, 4, 128), (16, 1, 256), (20, 2, 48), (3, 1, 16), (12, 1, 176)])
def test_large_queries_where_keys_are_zero(cuda_device, kv_type, spread, heads, kv_heads, dim):
    """Some dims of q are 2^spread times the others, and the keys have nothing there: the scores come from the others."""
    b = R.Batch([300, 1, 5000, 64], kv_heads, dim, 16, seed=34)
    q = queries(b, heads, 34, gain=3.0)
    wide = [0, 5] if spread % 2 else [dim - 1]
    g = q.view(len(b.lens), heads, dim)
    g[..., wide] *= 2.0 ** spread
    g[2, :, 1] = 0
    for k in b.k:
        k[..., wide] = 0
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        hold(b, kv_type, q, attend(c, q)[0])
        small = (q.float() * 2.0 ** -80).to(torch.bfloat16)  # (and far from 1: the scale brings it back)
        for i, n in enumerate(b.lens):
            assert torch.equal(small[i].double() * 2.0 ** 80, q[i].double())
        out = attend(c, small, scale=dim ** -0.5 * 2.0 ** 80)[0]
        hold(b, kv_type, q, out)


@pytest.mark.parametrize("kv_type", ["e4m3", "int8"])
@pytest.mark.parametrize("spread", [3, 25])
def test_every_code_of_a_key(cuda_device, kv_type, spread):
    """Keys of all codes, the lowest of a row's range among them, whose largest meets a q of 0."""
    dim = 128
    b = R.Batch([256, 40], 1, dim, 16, seed=35)
    codes = torch.arange(1, 128).double()
    if kv_type == "e4m3":
        codes = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 2^-9 to 448
    g = torch.Generator().manual_seed(35)
    for k in b.k:
        pick = codes[torch.randint(len(codes), k.shape, generator=g)]
        pick[::2] = codes[torch.randint(7, pick[::2].shape, generator=g)]
        pick = pick * (torch.randint(2, k.shape, generator=g) * 2 - 1)
        pick[..., 9] = R.QMAX[kv_type]
        pick[..., 3] = 0
        k.copy_((pick / 16).to(torch.bfloat16))
    q = queries(b, 4, 35, gain=0.5)
    v = q.view(2, 4, dim)
    v[..., 9] = 0
    v[..., 3] *= 2.0 ** spread
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        hold(b, kv_type, q, attend(c, q)[0])


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("size", [1, 10, 14, 20, 30, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_one_token_takes_all_whatever_its_score(cuda_device, kv_type, size, sign):
    """Scores of 2^size and far apart: the result is the top token's value, which no error of a score touches: rounded
    to bf16, its weight to fp16 over an 8-bit cache (2^-11), and 2^-15 for exponential and logarithm."""
    heads, dim, top = 8, 64, [0, 100, 4999, 7]
    b = R.Batch([1, 300, 5000, 40], 2, dim, 16, seed=36)
    q = torch.zeros(4, heads, dim)
    q[..., 5] = 2.0 ** (size / 2)
    q[..., 9] = 2.0 ** (size / 2 - 20)
    q = q.view(4, -1).to(torch.bfloat16)
    for i, (k, v) in enumerate(zip(b.k, b.v)):
        k.zero_()
        k[..., 5] = sign * 2.0 ** (size / 2) * (0.25 if sign > 0 else 4.0)
        k[top[i], :, 5] = sign * 2.0 ** (size / 2)
        v[::3] *= 2.0 ** -30
        v[1::3] *= 2.0 ** 30
    scale = 200.0 if size < 10 else 1.0
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        out, lse = attend(c, q, scale=scale)
        for i, n in enumerate(b.lens):
            want = R.values(b.v[i][top[i]], kv_type).repeat_interleave(heads // 2, 0)
            got = out[i].view(heads, dim).double()
            assert ((got - want).abs() <= want.abs() * (R.U_BF16 + 2.0 ** -11 + 2.0 ** -15)).all(), "sequence %d" % i
        assert c.error() == 0


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_values_near_the_end_of_the_range(cuda_device, kv_type):
    """One token has V of 2^127 and a score a few bits above those before it, the others have none: weights are never
    above 1, so that nothing passes the range on the way to a result inside it."""
    n = 200000  # several steps for each warp: the token is the first of its warp's at few of the places
    b = R.Batch([n], 1, 64, 64, seed=37)
    q = torch.zeros(1, 4, 64)
    q[..., 0] = 8.0
    q = q.view(1, -1).to(torch.bfloat16)
    b.k[0].zero_()
    b.v[0].zero_()
    with Cache(b, kv_type, cuda_device) as c:
        for at in (70001, 100000, 100064, 100129, 100200, 100260, 199999):
            for score in (0.5, 2.5):
                b.k[0][at, 0, 0] = score
                b.v[0][at] = torch.where(torch.arange(64) % 2 == 0, 2.0 ** 127, -1.5 * 2.0 ** 126).to(torch.bfloat16)
                c.append()
                out, lse = attend(c, q)
                hold(b, kv_type, q, out)
                b.k[0][at] = 0
                b.v[0][at] = 0
        assert c.error() == 0
