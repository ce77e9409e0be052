"""The operators around the adapted projections of a decode step, as they are measured.

A step of a served model runs, per layer: the residual's addition and root-mean-square
norm that make the rows ``lora_linear`` / ``lora_apply`` read (``lora_rmsnorm``), the
adapted q/k/v projections, the new tokens' keys and values quantised into the paged
cache (``lora_kv_append``), attention of one new token over that cache
(``lora_attend``), and the adapted output projection.  A prefill chunk appends many
rows and reads the whole prefix back (``lora_kv_append``, ``lora_kv_gather``).

Three kinds of case:
  norm    T rows of `width`: h = x + residual, h kept, h / rms(h) * weight as bf16
          and as e4m3 with a scale per row or per group of columns
  chunk   new rows of several sequences into the cache, then each sequence's whole
          prefix (old and new rows) back as bf16
  decode  one new row per sequence into the cache, then its attention over the cache

``own`` false computes them in elementary torch operations, true through the library.
"""

import math
import random

import torch

own = False

E4M3_MAX, INT8_MAX = 448.0, 127.0
EPS = 1e-5


# ------------------------------------------------------------------ cases


def _norm(name, rows, width, group):
    return {"name": name, "kind": "norm", "rows": rows, "width": width, "group": group}


def _chunk(name, seqs, rows, lo, hi, kv_heads, dim, type, page, mix):
    return {"name": name, "kind": "chunk", "seqs": seqs, "rows": rows, "lo": lo, "hi": hi, "kv_heads": kv_heads,
            "dim": dim, "type": type, "page": page, "mix": mix}


def _decode(name, seqs, lo, hi, heads, kv_heads, dim, type, page, mix, window=0, sinks=False, padded=0, empty=0):
    return {"name": name, "kind": "decode", "seqs": seqs, "lo": lo, "hi": hi, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "type": type, "page": page, "mix": mix, "window": window, "sinks": sinks, "padded": padded,
            "empty": empty}


def listed():
    return [
        # one request's token between two layers of a 4096-wide model: latency alone
        _norm("norm_token", 1, 4096, 0),
        # the decode batch of 512 rows, one scale per row (a row-scaled 8-bit base product)
        _norm("norm_batch", 512, 4096, 0),
        # a ragged batch at width 2880 with a scale for every 32 columns
        _norm("norm_ragged", 333, 2880, 32),
        # a prefill batch with a scale for every 128 columns (block-scaled 8-bit base product)
        _norm("norm_prefill", 8192, 4096, 128),
        # a prefill batch of 8 segments with Zipf lengths over cached prefixes, 32 heads of 128
        _chunk("chunk_e4m3", 8, 4096, 200, 3000, 32, 128, "e4m3", 64, 11),
        # a few short continuations at odd lengths, 8 heads of 64
        _chunk("chunk_int8", 5, 173, 1, 700, 8, 64, "int8", 16, 12),
        # 16 short requests on a 256-wide model: the smallest step, latency alone
        _decode("decode_tiny", 16, 1, 100, 8, 8, 32, "bf16", 16, 13),
        # the 64-request decode batch with 32 heads of 128, each with its own keys and values
        _decode("decode_mha", 64, 200, 4000, 32, 32, 128, "bf16", 16, 14),
        # one request with a very long context: the cache's length has to be split
        _decode("decode_long", 1, 131071, 131071, 32, 8, 128, "bf16", 64, 15),
        # the 512-request decode batch, 4 query heads to a key head, 8-bit cache, a padded tail
        _decode("decode_batch", 512, 64, 2048, 32, 8, 128, "e4m3", 32, 16, padded=17),
        # sliding-window layer with attention sinks, 8 query heads of 64 to a key head
        _decode("decode_window", 256, 1, 8000, 64, 8, 64, "int8", 16, 17, window=128, sinks=True, empty=3),
        # wide heads, 16 query heads to a key head, odd lengths
        _decode("decode_wide", 37, 5, 9001, 32, 2, 256, "int8", 128, 18),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heavy(c):
    """Whether a case moves or computes more, or holds more of a cache, than the largest listed one."""
    most = [work(x) for x in listed()]
    w = work(c)
    held = c["seqs"] * c["hi"] * c["kv_heads"] * c["dim"] if c["kind"] != "norm" else 0
    return w["bytes"] > max(x["bytes"] for x in most) or w["flops"] > max(x["flops"] for x in most) or held > 1 << 30


def draw(rng):
    kind = rng.choice(["norm", "chunk", "decode", "decode"])
    if kind == "norm":
        group = rng.choice([0, 0, 32, 64, 128])
        width = max(1, _log(rng, 64, 16384) // max(group, 8)) * max(group, 8)
        c = _norm("", _log(rng, 1, 8192), width, group)
        while _heavy(c):
            c["rows"] //= 2
        del c["name"]
        return c
    type = rng.choice(["bf16", "e4m3", "int8"])
    page = rng.choice([16, 16, 32, 64, 128])
    dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16, 32])
    mix = rng.randrange(1 << 30)
    if kind == "chunk":
        lo = rng.choice([0, 1, 100])
        c = _chunk("", _log(rng, 1, 64), _log(rng, 1, 4096), lo, max(lo + 1, _log(rng, 10, 4000)), kv_heads, dim, type,
                   page, mix)
    else:
        heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 12, 16, 32) if g * kv_heads <= 64])
        seqs, lo = _log(rng, 1, 512), rng.choice([1, 1, 17, 300])
        c = _decode("", seqs, lo, max(lo + 1, _log(rng, 20, 65536 if seqs < 8 else 8192)), heads, kv_heads, dim, type,
                    page, mix, window=rng.choice([0, 0, 0, 1, 100, 1024]), sinks=rng.random() < 0.25,
                    padded=seqs // 7 if rng.random() < 0.3 else 0, empty=seqs // 9 if rng.random() < 0.3 else 0)
    while _heavy(c):
        if c["hi"] > 2 * c["lo"] + 2:
            c["hi"] //= 2
        elif c["seqs"] > 1:
            c["seqs"] = (c["seqs"] + 1) // 2
            if kind == "decode":
                c["padded"], c["empty"] = c["padded"] // 2, c["empty"] // 2
        else:
            c["kv_heads"] = max(1, c["kv_heads"] // 2)
    del c["name"]
    return c


def _prefixes(case):
    """Lengths spread over the logarithm of lo .. hi, the last `padded` rows -1 (no request), `empty` of the others 0."""
    r = random.Random(case["mix"])
    lo, hi = case["lo"], case["hi"]
    n = [min(hi, max(lo, int((max(lo, 0.5)) * (hi / max(lo, 0.5)) ** r.random()))) for _ in range(case["seqs"])]
    if hi == lo:
        n = [lo] * case["seqs"]
    live = case["seqs"] - case.get("padded", 0)
    for i in r.sample(range(live), min(case.get("empty", 0), live)):
        n[i] = 0
    return n[:live] + [-1] * (case["seqs"] - live)


def _new_rows(case):
    """The chunk's new rows for each sequence: Zipf shares of the total, some of them none."""
    w = [(i + 1) ** -1.2 for i in range(case["seqs"])]
    n = [int(case["rows"] * x / sum(w)) for x in w]
    n[0] += case["rows"] - sum(n)
    random.Random(case["mix"] + 1).shuffle(n)
    return n


def _held(case):
    """Bytes of one token's key (or value) of one head in the cache."""
    return case["dim"] * 2 if case["type"] == "bf16" else case["dim"] + 4


def work(case):
    if case["kind"] == "norm":
        t, d, g = case["rows"], case["width"], case["group"]
        # x, residual, kept sum, bf16 output, 8-bit output; scales, weight
        return {"bytes": t * d * 9 + 4 * t * (d // g if g else 1) + 2 * d, "flops": 6 * t * d}
    h, d = case["kv_heads"], case["dim"]
    if case["kind"] == "chunk":
        old, new = sum(_prefixes(case)), case["rows"]
        # new rows read and written to the cache, old rows read from it, all rows out in bf16
        return {"bytes": 2 * h * (new * 2 * d + (new + old) * _held(case) + (new + old) * 2 * d),
                "flops": 4 * h * d * (2 * new + old)}
    n = [x for x in _prefixes(case)]
    live = sum(x > 0 for x in n)
    read = sum(min(x, case["window"] or x) for x in n if x > 0)
    rows = sum(x >= 0 for x in n)
    # the new row read (bf16) and written, the cache read, q in, out and lse written
    return {"bytes": 2 * h * (live * 2 * d + read * _held(case)) + case["heads"] * (live * 2 * d + rows * (2 * d + 4)),
            "flops": 4 * case["heads"] * d * read}


# ------------------------------------------------------------------ inputs


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _inputs(case, seed):
    """Everything random of a case, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["kind"] == "norm":
        t, d = case["rows"], case["width"]
        return {"x": _rand(gen, t, d), "residual": _rand(gen, t, d) * 3, "weight": 1 + _rand(gen, d) * 0.2}
    h, d = case["kv_heads"], case["dim"]
    # a few channels of the keys are several times larger than the others, as in trained models
    wide = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    wide[:: 16] = 4
    if case["kind"] == "chunk":
        old, new = _prefixes(case), _new_rows(case)
        lens = [a + b for a, b in zip(old, new)]
    else:
        lens = _prefixes(case)
        new = [int(x > 0) for x in lens]
        old = [max(x, 0) - b for x, b in zip(lens, new)]
    page = case["page"]
    pages = [-(-max(x, 0) // page) for x in lens]
    some = sum(pages) + 3
    order = torch.randperm(some, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = order[at:at + n]
        at += n
    s = {"lens": lens, "old": old, "new": new, "n_pages": some, "table": table.cuda(),
         "k_old": _rand(gen, sum(old), h * d) * wide.repeat(h), "v_old": _rand(gen, sum(old), h * d)}
    rows = case["rows"] if case["kind"] == "chunk" else len(lens)
    s["k"], s["v"] = _rand(gen, rows, h * d) * wide.repeat(h), _rand(gen, rows, h * d)
    if case["kind"] == "decode":
        s["q"] = _rand(gen, len(lens), case["heads"] * d)
        s["out"] = _rand(gen, len(lens), case["heads"] * d)  # what padded rows keep
        s["lse"] = torch.randn(len(lens), case["heads"], generator=gen, device="cuda")
        s["sinks"] = torch.randn(case["heads"], generator=gen, device="cuda") if case["sinks"] else None
    return s


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(counts):
    return _ints([0] + torch.tensor(counts).cumsum(0).tolist())


# ------------------------------------------------------------------ plain form


def _quantise(x, type):
    """x [..., dim] as held values and scales: codes x * qmax / amax rounded to the type, in 64 bits since the quotient
    often lies on the border of two codes; a row whose largest magnitude is under 2^-100 is held as zeros."""
    if type == "bf16":
        return x, None
    x = x.double()
    qmax = E4M3_MAX if type == "e4m3" else INT8_MAX
    amax = x.abs().amax(-1, keepdim=True)
    none = amax < 2.0 ** -100
    code = torch.where(none, 0, x * qmax / amax)
    scale = torch.where(none, 0, amax / qmax)[..., 0].float()
    if type == "e4m3":
        return code.clamp(-qmax, qmax).to(torch.float8_e4m3fn).view(torch.uint8), scale
    return code.round().clamp(-qmax, qmax).to(torch.int8), scale


def _values(held, scale):
    """The fp32 values that held codes stand for."""
    if held.dtype == torch.bfloat16:
        return held.float()
    if held.dtype == torch.uint8:
        held = held.view(torch.float8_e4m3fn)
    return held.float() * scale[..., None]


def _slots(table, page, seq, pos):
    return table[seq, pos // page].long() * page + pos % page


def _plain_cache(case, s):
    """Both caches as [slots, heads, dim] with the old rows in place, and where the new rows go."""
    n, h, d = s["n_pages"] * case["page"], case["kv_heads"], case["dim"]
    rows = lambda counts, start: (  # noqa: E731
        torch.cat([torch.full((c,), i) for i, c in enumerate(counts)]).cuda(),
        torch.cat([torch.arange(b, b + c) for b, c in zip(start, counts)]).cuda())
    zero = [0] * len(s["lens"])
    old, new = _slots(s["table"], case["page"], *rows(s["old"], zero)), _slots(s["table"], case["page"], *rows(s["new"], s["old"]))
    p = {"new_at": new, "all_at": _slots(s["table"], case["page"], *rows([max(x, 0) for x in s["lens"]], zero)),
         "new_rows": torch.tensor(s["new"], device="cuda").nonzero()[:, 0] if case["kind"] == "decode" else None,
         "lens_gpu": torch.tensor(s["lens"], device="cuda")}
    for name in ("k", "v"):
        held, scale = _quantise(s.pop(name + "_old").view(-1, h, d), case["type"])
        p[name + "_held"] = torch.zeros(n, h, d, dtype=held.dtype, device="cuda").index_copy_(0, old, held)
        p[name + "_scale"] = None if scale is None else torch.zeros(n, h, device="cuda").index_copy_(0, old, scale)
    return p


def _plain_write(s, name):
    c = s["case"]
    x = s[name].view(-1, c["kv_heads"], c["dim"])
    held, scale = _quantise(x if s["new_rows"] is None else x[s["new_rows"]], c["type"])
    s[name + "_held"][s["new_at"]] = held
    if scale is not None:
        s[name + "_scale"][s["new_at"]] = scale


def _plain_read(s, name, at):
    scale = s[name + "_scale"]
    return _values(s[name + "_held"][at], None if scale is None else scale[at])


def _plain_attend(s):
    c, lens = s["case"], s["lens_gpu"]
    n, h, d = c["seqs"], c["kv_heads"], c["dim"]
    most = max(1, max(s["lens"]))
    span = min(most, c["window"] or most)  # the last `span` positions of each sequence
    pos = lens[:, None] - span + torch.arange(span, device="cuda")
    seen = (pos >= 0) & (lens[:, None] > 0)
    at = torch.where(seen, _slots(s["table"], c["page"], torch.arange(n, device="cuda")[:, None], pos.clamp(min=0)), 0)
    k, v = _plain_read(s, "k", at), _plain_read(s, "v", at)
    q = s["q"].float().view(n, h, -1, d)
    score = torch.einsum("nhgd,nlhd->nhgl", q, k) / math.sqrt(d)
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1)
    sink = s["sinks"].view(1, h, -1) if s["sinks"] is not None else None
    if sink is not None:
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0, top)
    p = torch.exp(score - top[..., None])
    total = p.sum(-1)
    if sink is not None:
        total = total + torch.exp(sink - top)
    out = torch.einsum("nhgl,nlhd->nhgd", p, v) / torch.where(total == 0, 1, total)[..., None]
    keep = (lens < 0)[:, None]
    return {"out": torch.where(keep, s["out"], out.reshape(n, -1).to(torch.bfloat16)),
            "lse": torch.where(keep, s["lse"], (top + total.log()).reshape(n, -1))}


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    inv = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = h * inv * s["weight"].float()
    t, d = y.shape
    code, scale = _quantise(y.view(t, d // (s["case"]["group"] or d), -1), "e4m3")
    return {"sum": h.to(torch.bfloat16), "y": y.to(torch.bfloat16),
            "q": code.view(torch.float8_e4m3fn).reshape(t, d), "scale": scale if s["case"]["group"] else scale[:, 0]}


# ------------------------------------------------------------------ the library


def _own_state(case, s):
    """What a serving program keeps: output buffers, the cache with the old rows in it, workspace."""
    import adapter_deltas_b200 as L

    s["L"] = L
    if case["kind"] == "norm":
        t, d, g = case["rows"], case["width"], case["group"]
        s["sum"], s["y"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["q"] = torch.empty(t, d, dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.empty(t, d // g, device="cuda") if g else torch.empty(t, device="cuda")
        return s
    type = {"bf16": L.LORA_KV_BF16, "e4m3": L.LORA_KV_E4M3, "int8": L.LORA_KV_INT8}[case["type"]]
    shape = (1, s["n_pages"], case["page"], case["kv_heads"], case["dim"], type)
    mem = torch.empty(L.lora_kv_bytes_required(*shape), dtype=torch.uint8, device="cuda")
    s["kv"] = L.lora_kv_create(torch.cuda.current_device(), *shape, mem)
    if sum(s["old"]):
        L.lora_kv_append(s["kv"], 0, s["k_old"], s["v_old"], s["table"], _ints(s["old"]), _offsets(s["old"]))
    del s["k_old"], s["v_old"]
    s["lens_gpu"] = _ints(s["lens"])
    if case["kind"] == "chunk":
        s["new_offsets"], s["all_offsets"] = _offsets(s["new"]), _offsets(s["lens"])
        s["k_out"] = torch.empty(sum(s["lens"]), case["kv_heads"] * case["dim"], dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        s["ws"] = torch.empty(L.lora_attend_workspace_bytes(s["kv"], case["heads"]), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        return _own_state(case, s)
    if case["kind"] != "norm":
        s.update(_plain_cache(case, s))
    return s


def run(s):
    kind = s["case"]["kind"]
    if own:
        L = s["L"]
        if kind == "norm":
            L.lora_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["sum"], y=s["y"], q=s["q"],
                           q_scales=s["scale"])
            return {"sum": s["sum"], "y": s["y"], "q": s["q"], "scale": s["scale"]}
        if kind == "chunk":
            L.lora_kv_append(s["kv"], 0, s["k"], s["v"], s["table"], s["lens_gpu"], s["new_offsets"])
            L.lora_kv_gather(s["kv"], 0, s["k_out"], s["v_out"], s["table"], s["lens_gpu"], s["all_offsets"])
            return {"k": s["k_out"], "v": s["v_out"]}
        L.lora_kv_append(s["kv"], 0, s["k"], s["v"], s["table"], s["lens_gpu"])
        L.lora_attend(s["kv"], 0, s["q"], s["out"], s["table"], s["lens_gpu"], s["ws"], window=s["case"]["window"],
                      sinks=s["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "norm":
        return _plain_norm(s)
    _plain_write(s, "k")
    _plain_write(s, "v")
    if kind == "chunk":
        width = s["case"]["kv_heads"] * s["case"]["dim"]
        return {n: _plain_read(s, n, s["all_at"]).to(torch.bfloat16).view(-1, width) for n in ("k", "v")}
    return _plain_attend(s)


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_held(x, type):
    """Values in 64 bits that a cache of this type holds for rows x [..., dim]."""
    x = x.double()
    if type == "bf16":
        return x
    most = x.abs().amax(-1, keepdim=True)
    top = E4M3_MAX if type == "e4m3" else INT8_MAX
    code = x * top / most  # (x * top is exact, so a tie stays one)
    step = torch.ones_like(code)
    if type == "e4m3":  # 3 bits after the leading one, the lowest exponent -6
        step = torch.exp2((torch.frexp(code).exponent - 1).clamp(min=-6).double() - 3)
    code = (torch.round(code / step) * step).clamp(-top, top)
    return torch.where(most < 2.0 ** -100, 0.0, code * most / top)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "norm":
        h = s["x"].double() + s["residual"].double()
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
        t, d = y.shape
        g = case["group"] or d
        blocks = y.view(t, -1, g)
        unit = blocks.abs().amax(-1) / E4M3_MAX
        code = _exact_held(blocks, "e4m3") / torch.where(unit == 0, 1, unit)[..., None]
        return {"sum": h, "y": y, "q": code.view(t, d), "scale": unit if case["group"] else unit[:, 0]}
    h, d = case["kv_heads"], case["dim"]
    olds, news = [torch.tensor(s[n]).cumsum(0).tolist() for n in ("old", "new")]
    outs = {"k": [], "v": [], "out": [], "lse": []}
    for i, length in enumerate(s["lens"]):
        both = {}
        for n in ("k", "v"):
            fresh = s[n][news[i] - s["new"][i]:news[i]] if case["kind"] == "chunk" else s[n][i:i + s["new"][i]]
            both[n] = torch.cat([s[n + "_old"][olds[i] - s["old"][i]:olds[i]], fresh]).view(-1, h, d)
        if case["kind"] == "chunk":
            for n in ("k", "v"):
                outs[n].append(_exact_held(both[n], case["type"]).view(-1, h * d))
            continue
        if length < 0:
            outs["out"].append(s["out"][i].double())
            outs["lse"].append(s["lse"][i].double())
            continue
        first = max(0, length - case["window"]) if case["window"] else 0
        k, v = (_exact_held(both[n][first:], case["type"]).transpose(0, 1) for n in ("k", "v"))
        score = s["q"][i].double().view(h, -1, d) @ k.transpose(1, 2) / math.sqrt(d)
        if s["sinks"] is not None:
            score = torch.cat([score, s["sinks"].double().view(h, -1, 1)], -1)
        lse = torch.logsumexp(score, -1)
        share = torch.exp(score - lse[..., None])[..., :k.shape[1]] if score.shape[-1] else score
        outs["out"].append((share @ v).reshape(-1))
        outs["lse"].append(lse.reshape(-1))
    if case["kind"] == "chunk":
        return {n: torch.cat(outs[n]) for n in ("k", "v")}
    return {n: torch.stack(outs[n]) for n in ("out", "lse")}
