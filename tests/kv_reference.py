"""Plain 64-bit definitions of the key/value cache, the attention over it and
the norm, and the error bounds that the tests hold the kernels to."""

from __future__ import annotations

import math

import torch

U_BF16, U_FP32 = 2.0 ** -8, 2.0 ** -24  # half a step of each type, relative
TYPES = {"bf16": 0, "e4m3": 1, "int8": 2}
QMAX = {"e4m3": 448.0, "int8": 127.0}


def round_e4m3(x: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value (ties to even) of doubles of magnitude at most 448."""
    e = (torch.frexp(x).exponent - 1).clamp(min=-6)
    step = torch.exp2(e.double() - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def held(x: torch.Tensor, kv_type: str):
    """bf16 rows [..., dim] as (codes, fp32 scale), both as doubles; bf16: the rows and 1."""
    x = x.double()
    if kv_type == "bf16":
        return x, torch.ones(x.shape[:-1], dtype=torch.float64)
    amax = x.abs().amax(-1, keepdim=True)
    none = amax < 2.0 ** -100
    ratio = torch.where(none, 0.0, x * QMAX[kv_type] / torch.where(none, 1.0, amax))  # (x * qmax is exact)
    code = round_e4m3(ratio) if kv_type == "e4m3" else torch.round(ratio).clamp(-127, 127)
    scale = torch.where(none, 0.0, amax / QMAX[kv_type])[..., 0].float().double()
    return code, scale


def values(x: torch.Tensor, kv_type: str) -> torch.Tensor:
    code, scale = held(x, kv_type)
    return code * scale[..., None]


def read_back(x: torch.Tensor, kv_type: str) -> torch.Tensor:
    """The bf16 rows that a read-back returns: the fp32 product code * scale, rounded once more."""
    if kv_type == "bf16":
        return x
    code, scale = held(x, kv_type)
    return (code.float() * scale.float()[..., None]).to(torch.bfloat16)


def attend(q, k, v, kv_type, scale, window=0, sinks=None):
    """One sequence: q [heads, dim], k / v [len, kv_heads, dim] bf16.  Returns out, lse and what each may be off by.

    A score is a sum of dim products in fp32: off by at most (dim + 4) rounding
    steps (2^-23 each, the tensor cores truncate) of the sum of magnitudes,
    times the scale.  A weight is off by that much relatively (twice: itself
    and the denominator), plus 2^-15 for the exponential, the running rescale
    and its split into two bf16 terms, plus len * 2^-23 for the sums; the result
    is rounded to bf16 once.

    With an 8-bit cache q is split into 8-bit terms, which leaves at most 2^-22 of
    a head's largest |q| per dim: within the dim + 4 steps above.  The weights
    times V's scales are rounded to fp16 (2^-11 relative), in units of 2^-9 of the
    largest scale u (or less): a small one may be off by half of fp16's smallest
    step, 2^-25 * 2^-9 u = 2^-34 u, and the sum over len tokens of codes c by
    len * 2^-34 u max|c| (weights are relative to one of the scores, so that the
    denominator is at least 1).
    """
    heads, dim = q.shape
    kv_heads = k.shape[1]
    n = k.shape[0]
    if window and n > window:
        k, v = k[n - window:], v[n - window:]
    kx, vx = values(k, kv_type).transpose(0, 1), values(v, kv_type).transpose(0, 1)  # [kv_heads, len, dim]
    qx = q.double().view(kv_heads, -1, dim)
    s = scale * qx @ kx.transpose(1, 2)
    mag = (abs(scale) * qx.abs() @ kx.abs().transpose(1, 2)).amax(-1) if kx.shape[1] else torch.zeros(s.shape[:2]).double()
    full = s if sinks is None else torch.cat([s, sinks.double().view(kv_heads, -1, 1)], -1)
    lse = torch.logsumexp(full, -1) if full.shape[-1] else torch.full(s.shape[:2], -math.inf, dtype=torch.float64)
    p = torch.exp(s - lse[..., None]) if s.shape[-1] else s
    out, spread = p @ vx, p @ vx.abs()
    err_s = mag * (dim + 4) * 2.0 ** -23
    rel = 2 * err_s + 2.0 ** -15 + kx.shape[1] * 2.0 ** -23
    if kv_type != "bf16":
        rel = rel + 2.0 ** -11
    tol_out = U_BF16 * out.abs() + rel[..., None] * spread * (1 + U_BF16) + 1e-38
    if kv_type != "bf16" and len(v):
        code, u = held(v, kv_type)
        floor = code.abs().amax((0, 2)) * u.nan_to_num().amax(0) * len(v) * 2.0 ** -34  # [kv_heads]
        tol_out = tol_out + floor[:, None, None]
    tol_lse = err_s + (kx.shape[1] + 8) * 2.0 ** -23 + lse.abs().nan_to_num(posinf=0) * 2.0 ** -22
    return out.reshape(heads, dim), lse.reshape(heads), tol_out.reshape(heads, dim), tol_lse.reshape(heads)


def norm(x, residual, weight, eps):
    h = x.double() + (residual.double() if residual is not None else 0)
    return h, h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * weight.double()


class Batch:
    """Sequences with scattered pages and their bf16 keys and values, on the CPU."""

    def __init__(self, lens, kv_heads, dim, page, seed=0, spare=3, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.kv_heads, self.dim, self.page = list(lens), kv_heads, dim, page
        need = [-(-max(n, 0) // page) for n in self.lens]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(self.lens), max(1, max(need, default=1))), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.k = [(torch.randn(max(n, 0), kv_heads, dim, generator=g) * gain).to(torch.bfloat16) for n in self.lens]
        self.v = [torch.randn(max(n, 0), kv_heads, dim, generator=g).to(torch.bfloat16) for n in self.lens]

    def rows(self, counts=None):
        """Row offsets and the concatenated last counts[s] tokens of each sequence (all by default)."""
        counts = [max(n, 0) for n in self.lens] if counts is None else counts
        off = torch.tensor([0] + list(torch.tensor(counts, dtype=torch.int64).cumsum(0)), dtype=torch.int32)
        width = self.kv_heads * self.dim
        cat = lambda t: torch.cat([x[len(x) - c:].reshape(c, width) for x, c in zip(t, counts)])  # noqa: E731
        return off, cat(self.k), cat(self.v)
