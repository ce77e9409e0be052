"""Attention of one new token per sequence over the paged cache, against the
definition in 64 bits on the values the cache holds, within bounds derived
from the roundings (kv_reference.attend)."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R
from test_gpu_kv import Cache

pytestmark = pytest.mark.gpu


def attend(c, q, window=0, sinks=None, scale=None, lens=None, want_lse=True, ws=None, fill=7.0):
    dev = c.device
    heads = q.shape[1] // c.b.dim
    q = q.to(dev)
    out = torch.full_like(q, fill)
    lse = torch.full((q.shape[0], heads), fill, device=dev) if want_lse else None
    ws = torch.full((L.lora_attend_workspace_bytes(c.kv, heads),), 255, dtype=torch.uint8, device=dev) if ws is None else ws
    L.lora_attend(c.kv, 0, q, out, c.table, c.lens if lens is None else lens, ws, scale=scale, window=window,
                  sinks=None if sinks is None else sinks.to(dev), lse=lse)
    return out.cpu(), lse.cpu() if want_lse else None


def check(c, kv_type, q, out, lse, window=0, sinks=None, scale=None, fill=7.0):
    dim = c.b.dim
    for i, n in enumerate(c.b.lens):
        if n < 0:
            assert (out[i] == fill).all() and (lse is None or (lse[i] == fill).all())
            continue
        o, l, to, tl = R.attend(q[i].view(-1, dim), c.b.k[i], c.b.v[i], kv_type, dim ** -0.5 if scale is None else scale,
                                window, sinks)
        got = out[i].view(-1, dim).double()
        off = ((got - o).abs() / to).max() if torch.isfinite(got).all() else float("nan")
        assert off <= 1, "sequence %d of length %d: %s of what it may be off" % (i, n, off)
        if lse is not None:
            x = lse[i].double()
            same = (x == l) | ((x - l).abs() <= tl)
            assert same.all(), "sequence %d of length %d: lse off by %s" % (i, n, (x - l).abs().max())
    assert c.error() == L.LORA_OK


def queries(b, heads, seed, gain=1.0):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(len(b.lens), heads * b.dim, generator=g) * gain).to(torch.bfloat16)


CASES = [  # heads, kv_heads, dim, page, lens
    (8, 8, 128, 16, [1, 2, 15, 16, 17, 31, 32, 33, 100]),
    (32, 8, 128, 64, [1, 1000, 63, 64, 65]),
    (64, 8, 64, 16, [129, 1, 300, 77]),
    (4, 4, 16, 16, [5, 50]),
    (10, 5, 80, 16, [40, 111]),
    (12, 4, 96, 128, [130, 260]),
    (24, 2, 256, 16, [18, 100]),
    (16, 1, 208, 1024, [1030]),
    (9, 1, 48, 32, [70] * 20),
    (40, 2, 32, 16, [200, 33]),
    (64, 1, 128, 16, [500, 3]),
    (6, 3, 112, 32, [95]),
    (14, 2, 160, 64, [200, 64, 1]),
]


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens", CASES)
def test_against_the_definition(cuda_device, kv_type, heads, kv_heads, dim, page, lens):
    b = R.Batch(lens, kv_heads, dim, page, seed=heads + dim)
    q = queries(b, heads, dim)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q))


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 5000])
def test_window(cuda_device, kv_type, window):
    b = R.Batch([1, 14, 16, 17, 33, 116, 117, 400, 0, -1], 2, 64, 32, seed=window)
    q = queries(b, 8, window)
    sinks = torch.randn(8, generator=torch.Generator().manual_seed(window))
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q, window=window), window=window)
        check(c, kv_type, q, *attend(c, q, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_empty_and_padded_rows(cuda_device, kv_type):
    b = R.Batch([0, -1, 5, 0, 200, -1, 0, -1], 4, 64, 16, seed=1)
    q = queries(b, 8, 1)
    sinks = torch.linspace(-2, 2, 8)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        out, lse = attend(c, q)
        assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
        check(c, kv_type, q, out, lse)
        out, lse = attend(c, q, sinks=sinks)
        assert torch.equal(lse[0], sinks)
        check(c, kv_type, q, out, lse, sinks=sinks)
        out, _ = attend(c, q, want_lse=False)
        check(c, kv_type, q, out, None)
    b = R.Batch([-1] * 300, 1, 32, 16)
    with Cache(b, kv_type, cuda_device) as c:
        q = queries(b, 4, 2)
        out, lse = attend(c, q)
        assert (out == 7.0).all() and (lse == 7.0).all()
        c.lens.zero_()
        out, lse = attend(c, q)
        assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_many_short_and_few_long(cuda_device, kv_type):
    """More sequences than blocks, with lengths from none to long, and one sequence cut over all of them."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(-1, 60, (700,), generator=g).tolist()
    lens[5], lens[699] = 3001, 1111
    b = R.Batch(lens, 2, 32, 16, seed=2)
    q = queries(b, 4, 3)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q))
    b = R.Batch([40000], 1, 64, 16, seed=3)
    q = queries(b, 8, 4)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q))
    b = R.Batch([2] * 3000 + [500], 1, 16, 16, seed=4)
    q = queries(b, 2, 5)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q))


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_large_scores(cuda_device, kv_type):
    """Scores in the hundreds: one token takes all the weight, and the maximum moves along the cache."""
    b = R.Batch([300, 70], 2, 128, 16, seed=6, gain=6.0)
    b.k[0] *= torch.linspace(0.2, 3, 300)[:, None, None].to(torch.bfloat16)
    q = queries(b, 8, 6, gain=8.0)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q))
        sinks = torch.tensor([1000.0, -1000.0, 0, 50, -50, 300, 1e30, -1e30])
        check(c, kv_type, q, *attend(c, q, sinks=sinks), sinks=sinks)
        check(c, kv_type, q, *attend(c, q, scale=0.001), scale=0.001)


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_a_value_that_is_not_finite_stays_with_its_head(cuda_device, kv_type):
    b = R.Batch([50, 50], 2, 64, 16, seed=7)
    b.v[0][20, 1, 3] = float("nan")
    q = queries(b, 4, 7)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        out, _ = attend(c, q)
        out = out.view(2, 4, 64)
        assert torch.isnan(out[0, 2:, 3]).all()
        assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()
        # outside the window it is not seen
        out, _ = attend(c, q, window=29)
        assert torch.isfinite(out).all()


def test_strided_rows_and_equal_bits(cuda_device):
    b = R.Batch([77, 500, 3], 2, 64, 16, seed=8)
    q = queries(b, 8, 8)
    with Cache(b, "int8", cuda_device) as c:
        c.append()
        want, lse = attend(c, q)
        again, lse2 = attend(c, q)
        assert torch.equal(want, again) and torch.equal(lse, lse2)
        wide = torch.full((3, 1040), 7.0, dtype=torch.bfloat16, device=cuda_device)
        wide[:, 8:520] = q.to(cuda_device)
        out = wide[:, 528:]
        ws = torch.empty(L.lora_attend_workspace_bytes(c.kv, 8), dtype=torch.uint8, device=cuda_device)
        L.lora_attend(c.kv, 0, wide[:, 8:520], out, c.table, c.lens, ws)
        assert torch.equal(out.cpu(), want)
        assert (wide[:, :8] == 7).all() and (wide[:, 520:528] == 7).all()


def test_bad_lengths_and_pages(cuda_device):
    b = R.Batch([40, 40, 40], 2, 64, 16, seed=9)
    q = queries(b, 4, 9)
    with Cache(b, "bf16", cuda_device) as c:
        c.append()
        good, _ = attend(c, q)
        assert c.error() == L.LORA_OK
        for n in (49, -2, 1 << 30, -(1 << 31)):
            c.lens[1] = n
            out, lse = attend(c, q)
            assert c.error() == L.LORA_ERR_BAD_ID
            assert (out[1] == 7.0).all() and (lse[1] == 7.0).all()
            assert torch.equal(out[[0, 2]], good[[0, 2]])
        c.lens[1] = 40
        for page in (b.n_pages, -1, 1 << 30, -(1 << 31)):
            c.table[1, 1] = page
            out, _ = attend(c, q)
            assert c.error() == L.LORA_ERR_BAD_ID
            assert torch.equal(out[[0, 2]], good[[0, 2]])
            # the page's 16 tokens are left out
            keep = list(range(16)) + list(range(32, 40))
            o, _, tol, _ = R.attend(q[1].view(-1, 64), b.k[1][keep], b.v[1][keep], "bf16", 0.125)
            assert ((out[1].view(-1, 64).double() - o).abs() <= tol).all()


def test_a_batch_past_the_counters_is_reported(cuda_device):
    """64 sequences of 2^30 tokens that share one page, 1024 heads: past 2^30 steps an SM; nothing is attended to."""
    b = R.Batch([1, 0], 1024, 16, 1024, seed=15)
    with Cache(b, "bf16", cuda_device) as c:
        c.append()
        assert c.error() == L.LORA_OK
        lens = torch.full((66,), 1 << 30, dtype=torch.int32, device=cuda_device)
        lens[5], lens[6] = 0, -1
        table = torch.zeros(66, 1 << 20, dtype=torch.int32, device=cuda_device)
        q = torch.zeros(66, 1024 * 16, dtype=torch.bfloat16, device=cuda_device)
        out = torch.full_like(q, 7.0)
        ws = torch.empty(L.lora_attend_workspace_bytes(c.kv, 1024), dtype=torch.uint8, device=cuda_device)
        L.lora_attend(c.kv, 0, q, out, table, lens, ws)
        assert c.error() == L.LORA_ERR_BAD_ID
        keep = torch.arange(66) != 5
        assert (out[5] == 0).all() and (out.cpu()[keep] == 7.0).all()
        few = queries(b, 1024, 15)
        check(c, "bf16", few, *attend(c, few, ws=ws))


def test_refusals(cuda_device):
    b = R.Batch([20, 20], 2, 64, 16, seed=10)
    q = queries(b, 4, 10).to(cuda_device)
    with Cache(b, "bf16", cuda_device) as c:
        out, lse = torch.empty_like(q), torch.empty(2, 4, device=cuda_device)
        ws = torch.empty(L.lora_attend_workspace_bytes(c.kv, 4), dtype=torch.uint8, device=cuda_device)
        assert all(L.lora_attend_workspace_bytes(c.kv, n) == 0 for n in (3, 0, -2, 4098))

        def code(layer=0, q=q, out=out, table=c.table, lens=c.lens, ws=ws, **more):
            with pytest.raises((L.LoraError, ValueError)) as e:
                L.lora_attend(c.kv, layer, q, out, table, lens, ws, **more)
            return getattr(e.value, "code", None)

        n = L.lora_kernel_launches()
        assert code(layer=1) == L.LORA_ERR_INVALID_ARG
        assert code(q=q[:, :192], out=out[:, :192]) == L.LORA_ERR_INVALID_ARG  # 3 heads over 2
        assert code(out=q) == L.LORA_ERR_INVALID_ARG
        assert code(ws=ws[:-1]) == L.LORA_ERR_WORKSPACE
        assert code(ws=torch.empty(ws.numel() + 16, dtype=torch.uint8, device=cuda_device)[8:]) == L.LORA_ERR_ALIGNMENT
        assert code(window=-1) == L.LORA_ERR_INVALID_ARG
        for scale in (0.0, -1.0, float("nan"), float("inf")):
            assert code(scale=scale) == L.LORA_ERR_INVALID_ARG
        code(q=q.float()), code(out=out[:1]), code(q=q[:, :100]), code(sinks=torch.zeros(3, device=cuda_device))
        code(lse=lse[:, :2]), code(lse=lse.double()), code(lens=c.lens.cpu()), code(table=c.table.float())
        wide = torch.zeros(2, 260, dtype=torch.bfloat16, device=cuda_device)
        assert code(q=wide[:, :256]) == L.LORA_ERR_ALIGNMENT
        assert L.lora_kernel_launches() == n


def test_streams_and_graphs(cuda_device):
    """Two calls at once on two streams, each with its workspace; a captured step replayed on new inputs."""
    b = R.Batch([900, 41, 0, 2000], 2, 64, 16, seed=11)
    q = queries(b, 8, 11)
    with Cache(b, "e4m3", cuda_device) as c:
        c.append()
        want, _ = attend(c, q)
        size = L.lora_attend_workspace_bytes(c.kv, 8)
        qd = q.to(cuda_device)
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [torch.zeros_like(qd) for _ in streams]
        wss = [torch.empty(size, dtype=torch.uint8, device=cuda_device) for _ in streams]
        torch.cuda.synchronize()
        for _ in range(20):
            for s, o, w in zip(streams, outs, wss):
                L.lora_attend(c.kv, 0, qd, o, c.table, c.lens, w, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(o.cpu(), want) for o in outs)

        out = torch.zeros_like(qd)
        k = torch.zeros(4, 128, dtype=torch.bfloat16, device=cuda_device)
        v = torch.zeros_like(k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lora_kv_append(c.kv, 0, k, v, c.table, c.lens)
            L.lora_attend(c.kv, 0, qd, out, c.table, c.lens, wss[0])
        for lens in ([900, 41, 0, 2000], [17, -1, 0, 1], [1, 33, 0, 1999]):
            c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            for i, n in enumerate(lens):
                if n > 0:
                    k[i], v[i] = b.k[i][n - 1].view(-1).to(cuda_device), b.v[i][n - 1].view(-1).to(cuda_device)
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            whole = c.b
            cut = R.Batch([0] * 4, 2, 64, 16)
            cut.lens, cut.k, cut.v = lens, [x[:max(n, 0)] for x, n in zip(b.k, lens)], [x[:max(n, 0)] for x, n in zip(b.v, lens)]
            c.b = cut
            check(c, "e4m3", q, out.cpu(), None)
            c.b = whole


def test_waits_that_run_out(cuda_device):
    """Nothing is fetched: the launch completes, says so, leaves the rows, and the next call is right."""
    b = R.Batch([700, 33, -1, 5, 1200], 2, 64, 16, seed=12)
    q = queries(b, 8, 12)
    with Cache(b, "bf16", cuda_device) as c:
        c.append()
        ws = torch.full((L.lora_attend_workspace_bytes(c.kv, 8),), 255, dtype=torch.uint8, device=cuda_device)
        want, _ = attend(c, q, ws=ws)
        out = torch.full_like(q.to(cuda_device), 7.0)
        L.lora_set_wait_limit_ns(2_000_000)
        try:
            L.lora_selftest_stalled_attend(c.kv, 0, q.to(cuda_device), out, c.table, c.lens, ws)
            torch.cuda.synchronize()
        finally:
            L.lora_set_wait_limit_ns(0)
        assert c.error() == L.LORA_ERR_TIMEOUT and c.error() == L.LORA_OK
        assert (out == 7.0).all()
        got, _ = attend(c, q, ws=ws)
        assert torch.equal(got, want) and c.error() == L.LORA_OK


@pytest.mark.parametrize("seed", range(10))
def test_random_batches(cuda_device, seed):
    """Lengths, head layouts and windows at random: every way of cutting a batch into blocks, warps and pieces."""
    g = torch.Generator().manual_seed(100 + seed)
    pick = lambda *v: v[int(torch.randint(len(v), (1,), generator=g))]  # noqa: E731
    kv_type = pick(*R.TYPES)
    kv_heads, group, dim = pick(1, 2, 3, 8), pick(1, 2, 4, 7, 8, 9, 16, 20), pick(16, 32, 64, 128, 144, 256)
    most = pick(20, 200, 3000)
    lens = (torch.rand(pick(1, 3, 40, 150), generator=g) ** 3 * most).int().tolist()
    for i in range(0, len(lens), 7):
        lens[i] = pick(-1, 0, lens[i], most)
    window, page = pick(0, 0, 1, 50, 300), pick(16, 32, 256)
    b = R.Batch(lens, kv_heads, dim, page, seed=seed)
    q = queries(b, kv_heads * group, seed)
    sinks = torch.randn(kv_heads * group, generator=g) if pick(True, False) else None
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q, window=window, sinks=sinks), window=window, sinks=sinks)


def test_one_workspace_for_caches_and_graphs_in_turn(cuda_device):
    """Calls that follow one another may share a workspace: two caches of different shapes, each in its graph."""
    batches = [R.Batch([1500, 3, 700], 2, 64, 16, seed=13), R.Batch([900, 900], 1, 128, 32, seed=14)]
    caches = [Cache(b, t, cuda_device) for b, t in zip(batches, ("int8", "bf16"))]
    try:
        qs = [queries(b, h, 13) for b, h in zip(batches, (8, 12))]
        size = max(L.lora_attend_workspace_bytes(c.kv, h) for c, h in zip(caches, (8, 12)))
        ws = torch.full((size,), 255, dtype=torch.uint8, device=cuda_device)
        graphs, outs = [], []
        for c, q in zip(caches, qs):
            c.append()
            qd, out = q.to(cuda_device), torch.zeros_like(q, device=cuda_device)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                L.lora_attend(c.kv, 0, qd, out, c.table, c.lens, ws)
            graphs.append((graph, qd)), outs.append(out)
        want = [attend(c, q)[0] for c, q in zip(caches, qs)]
        for turn in range(6):
            for out in outs:
                out.zero_()
            for graph, _ in graphs if turn % 2 else graphs[::-1]:
                graph.replay()
            if turn == 3:
                ws.random_(0, 255)  # whatever is written there in between does not matter
            torch.cuda.synchronize()
            assert all(torch.equal(o.cpu(), w) for o, w in zip(outs, want))
        for c, t, q, out in zip(caches, ("int8", "bf16"), qs, outs):
            check(c, t, q, out.cpu(), None)
    finally:
        for c in caches:
            c.__exit__()


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens", [(8, 2, 64, 64, [30000, 7, 20011]), (1, 1, 128, 16, [40000]),
                                                          (16, 1, 256, 32, [9000, 1, 5000]), (40, 5, 80, 16, [7777] * 3)])
def test_units_cut_over_many_blocks(cuda_device, kv_type, heads, kv_heads, dim, page, lens):
    """Joins of many parts, of two units in one block, and of fewer rows than threads."""
    b = R.Batch(lens, kv_heads, dim, page, seed=17)
    q = queries(b, heads, 17)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        check(c, kv_type, q, *attend(c, q))
        check(c, kv_type, q, *attend(c, q, window=4097), window=4097)
