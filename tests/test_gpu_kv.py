"""The paged key/value cache: what is read back is bit for bit what the
definition in 64 bits holds, for every type, head layout, page size and way of
cutting the rows into calls."""

import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R

pytestmark = pytest.mark.gpu


class Cache:
    def __init__(self, b: R.Batch, kv_type: str, device, n_layers=1, n_pages=None):
        self.b = b
        shape = (n_layers, n_pages or b.n_pages, b.page, b.kv_heads, b.dim, R.TYPES[kv_type])
        # every byte 0xff: NaN in each of the types, so that whatever is read without having been written shows
        self.mem = torch.full((L.lora_kv_bytes_required(*shape),), 255, dtype=torch.uint8, device=device)
        self.kv = L.lora_kv_create(device.index, *shape, self.mem)
        self.table = b.table.to(device)
        self.lens = torch.tensor(b.lens, dtype=torch.int32, device=device)
        self.device = device

    def append(self, counts=None, lens=None, layer=0):
        off, k, v = self.b.rows(counts)
        lens = self.lens if lens is None else torch.tensor(lens, dtype=torch.int32, device=self.device)
        L.lora_kv_append(self.kv, layer, k.to(self.device), v.to(self.device), self.table, lens, off.to(self.device))

    def gather(self, counts=None, layer=0, fill=7.0):
        off, k, _ = self.b.rows(counts)
        ko = torch.full(k.shape, fill, dtype=torch.bfloat16, device=self.device)
        vo = torch.full(k.shape, fill, dtype=torch.bfloat16, device=self.device)
        L.lora_kv_gather(self.kv, layer, ko, vo, self.table, self.lens, off.to(self.device))
        return ko.cpu(), vo.cpu()

    def expect(self, kv_type, counts=None):
        _, k, v = self.b.rows(counts)
        shape = (-1, self.b.kv_heads, self.b.dim)
        return [R.read_back(x.view(shape), kv_type).view(x.shape) for x in (k, v)]

    def error(self):
        return L.lora_kv_get_error(self.kv)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        L.lora_kv_destroy(self.kv)


def same(got, want):
    """Equal values (the sign of a zero does not count: int8 has none)."""
    return all(torch.equal(g, w) for g, w in zip(got, want))


SHAPES = [  # kv_heads, dim, page, lens
    (8, 128, 16, [1, 15, 16, 17, 100]),
    (32, 128, 64, [333]),
    (2, 64, 32, [0, 5, -1, 64, 65]),
    (1, 16, 16, [40, 1]),
    (5, 80, 16, [33, 2]),
    (3, 96, 128, [129, 300]),
    (4, 256, 16, [18, 31]),
    (2, 192, 1024, [1030]),
    (7, 48, 32, [70] * 40),
    (1, 32, 16, [3] * 1500),
]


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("kv_heads,dim,page,lens", SHAPES)
def test_append_then_gather(cuda_device, kv_type, kv_heads, dim, page, lens):
    b = R.Batch(lens, kv_heads, dim, page, seed=dim + page)
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        assert same(c.gather(), c.expect(kv_type))
        # the last few tokens of each sequence alone
        some = [min(max(n, 0), 1 + i % 3) for i, n in enumerate(lens)]
        assert same(c.gather(some), c.expect(kv_type, some))
        assert c.error() == L.LORA_OK


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_decode_rows_and_chunks_agree(cuda_device, kv_type):
    """The same tokens written in one call, in chunks and one at a time leave the same bytes."""
    b = R.Batch([37, 18, 0, 53], 4, 64, 16, seed=3)
    images = []
    for way in ("whole", "chunks", "tokens"):
        with Cache(b, kv_type, cuda_device) as c:
            if way == "whole":
                c.append()
            else:
                step = 7 if way == "chunks" else 1
                for first in range(0, 53, step):
                    upto = [min(n, first + step) for n in b.lens]
                    counts = [max(0, u - min(n, first)) for u, n in zip(upto, b.lens)]
                    k = torch.cat([x[u - m:u].reshape(m, 256) for x, u, m in zip(b.k, upto, counts)]).to(cuda_device)
                    v = torch.cat([x[u - m:u].reshape(m, 256) for x, u, m in zip(b.v, upto, counts)]).to(cuda_device)
                    lens = torch.tensor([u if m else -1 for u, m in zip(upto, counts)], dtype=torch.int32)
                    if way == "tokens":  # one row per sequence; the rows of finished ones are skipped
                        full = torch.zeros(4, 256, dtype=torch.bfloat16, device=cuda_device)
                        kk, vv = full.clone(), full.clone()
                        at = torch.tensor(counts, device=cuda_device).bool()
                        kk[at], vv[at] = k, v
                        L.lora_kv_append(c.kv, 0, kk, vv, c.table, lens.to(cuda_device))
                    else:
                        off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
                        L.lora_kv_append(c.kv, 0, k, v, c.table, lens.to(cuda_device), off.to(cuda_device))
            assert same(c.gather(), c.expect(kv_type))
            assert c.error() == L.LORA_OK
            images.append(c.mem.cpu())
    assert torch.equal(images[0], images[1]) and torch.equal(images[0], images[2])


@pytest.mark.parametrize("kv_type", ["e4m3", "int8"])
def test_codes_at_the_borders(cuda_device, kv_type):
    """Quotients that lie half way between two codes, rows of zeros, the smallest and the largest magnitudes."""
    dim, rows = 64, []
    for amax in (1.0, 1.75, 3.5, 127.0, 224.0, 0.0078125, 2.0 ** 70, 3.3e38, 2.0 ** -99, 2.0 ** -100, 1e-35, 0.0):
        x = torch.linspace(-1, 1, dim).double() * amax
        rows.append(x.to(torch.bfloat16))
    m = torch.tensor([127.0] + [i + 0.5 for i in range(63)])          # int8 ties
    rows += [m.to(torch.bfloat16), (m * 2.0 ** -20).to(torch.bfloat16)]
    e = torch.tensor([448.0] + [1 + i / 16 for i in range(63)])       # e4m3 ties
    rows += [e.to(torch.bfloat16), (-e * 2.0 ** 40).to(torch.bfloat16)]
    b = R.Batch([len(rows)], 1, dim, 16)
    b.k = [torch.stack(rows)[:, None]]
    b.v = [torch.stack(rows).flip(0)[:, None]]
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        got, want = c.gather(), c.expect(kv_type)
        assert same(got, want), [(g - w).abs().amax(-1) for g, w in zip(got, want)]


@pytest.mark.parametrize("kv_type", ["e4m3", "int8"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_values_that_are_not_finite_read_back_as_nan(cuda_device, kv_type, bad):
    b = R.Batch([20], 2, 64, 16, seed=5)
    b.k[0][4, 1, 9] = bad
    with Cache(b, kv_type, cuda_device) as c:
        c.append()
        k, v = c.gather()
        k = k.view(20, 2, 64)
        assert torch.isnan(k[4, 1]).all()
        k[4, 1] = 0
        assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_rows_as_slices_of_a_fused_projection(cuda_device):
    b = R.Batch([9, 30], 2, 64, 16, seed=6)
    off, k, v = b.rows()
    fused = torch.zeros(39, 512, dtype=torch.bfloat16, device=cuda_device)
    fused[:, 256:384], fused[:, 384:] = k.to(cuda_device), v.to(cuda_device)
    with Cache(b, "e4m3", cuda_device) as c:
        L.lora_kv_append(c.kv, 0, fused[:, 256:384], fused[:, 384:], c.table, c.lens, off.to(cuda_device))
        both = torch.full((39, 264), 7.0, dtype=torch.bfloat16, device=cuda_device)
        L.lora_kv_gather(c.kv, 0, both[:, :128], both[:, 136:], c.table, c.lens, off.to(cuda_device))
        assert same((both[:, :128].cpu(), both[:, 136:].cpu()), c.expect("e4m3"))
        assert (both[:, 128:136] == 7.0).all()


@pytest.mark.parametrize("kv_type", list(R.TYPES))
@pytest.mark.parametrize("at,ld", [(0, 480), (8, 480), (16, 488), (24, 472), (16, 480)])
def test_rows_at_16_and_32_bytes(cuda_device, kv_type, at, ld):
    """Rows need start at multiples of 16 bytes only; where all start at 32 they are read and written 32 at a time."""
    b = R.Batch([33, 1, 70], 2, 80, 16, seed=16)
    off, k, v = b.rows()
    wide = torch.zeros(len(k), ld, dtype=torch.bfloat16)
    wide[:, at:at + 160], wide[:, at + 160:at + 320] = k, v
    src, dst = wide.to(cuda_device), torch.full(wide.shape, 7.0, dtype=torch.bfloat16, device=cuda_device)
    with Cache(b, kv_type, cuda_device) as c:
        cut = lambda t: (t[:, at:at + 160], t[:, at + 160:at + 320])  # noqa: E731
        L.lora_kv_append(c.kv, 0, *cut(src), c.table, c.lens, off.to(cuda_device))
        L.lora_kv_gather(c.kv, 0, *cut(dst), c.table, c.lens, off.to(cuda_device))
        assert same([x.cpu() for x in cut(dst)], c.expect(kv_type)) and c.error() == L.LORA_OK
        dst[:, at:at + 320] = 7.0
        assert (dst == 7.0).all()


def test_layers_and_far_pages(cuda_device):
    """Layers are apart, and pages beyond 4 GiB of the cache are reached."""
    b = R.Batch([40, 17], 8, 128, 16, seed=7)
    page_bytes = L.lora_kv_bytes_required(1, 1, 16, 8, 128, 0)
    n = (5 << 30) // page_bytes
    b.table = torch.where(b.table >= 0, n - 1 - b.table, b.table)
    with Cache(b, "bf16", cuda_device, n_layers=2, n_pages=n) as c:
        c.append(layer=1)
        low = c.mem[: n * page_bytes]
        assert (low[:: 4096] == 255).all() and (low[-page_bytes:] == 255).all()
        assert same(c.gather(layer=1), c.expect("bf16"))


def test_bad_lengths_pages_and_offsets_are_reported_and_skipped(cuda_device):
    b = R.Batch([20, 20, 20, 20], 2, 64, 16, seed=8)
    with Cache(b, "int8", cuda_device) as c:
        c.append()
        want = c.expect("int8")
        assert c.error() == L.LORA_OK
        # a page outside the cache, either side
        for page in (b.n_pages, -5):
            c.table[1, 1] = page
            before = c.mem.clone()
            c.append()
            assert torch.equal(before, c.mem) and c.error() == L.LORA_ERR_BAD_ID
            k, v = c.gather()
            assert c.error() == L.LORA_ERR_BAD_ID
            assert (k[36:40] == 7.0).all() and (v[36:40] == 7.0).all()
            keep = torch.ones(80, dtype=torch.bool)
            keep[36:40] = False
            assert same((k[keep], v[keep]), [w[keep] for w in want])
        c.table.copy_(b.table)
        # a length past the table, one below -1, one shorter than its rows
        for lens in ([20, 33, 20, 20], [20, 20, -2, 20], [20, 20, 20, 19]):
            before = c.mem.clone()
            c.append(lens=lens)
            assert c.error() == L.LORA_ERR_BAD_ID
            if lens[2] == -2:
                assert torch.equal(before, c.mem)
            c.append()
            assert c.error() == L.LORA_OK and torch.equal(before, c.mem)
        # offsets out of order or past the rows
        _, k, v = b.rows()
        lowest, highest = -(1 << 31), (1 << 31) - 1
        for off in ([0, 30, 20, 60, 80], [0, 20, 40, 60, 81], [-1, 20, 40, 60, 80], [lowest, highest, highest, highest, highest],
                    [lowest, lowest, -1, highest, highest], [highest, 20, 40, 60, lowest]):
            L.lora_kv_append(c.kv, 0, k.to(cuda_device), v.to(cuda_device), c.table, c.lens,
                             torch.tensor(off, dtype=torch.int32, device=cuda_device))
            assert c.error() == L.LORA_ERR_BAD_ID


def test_empty_calls_launch_nothing(cuda_device):
    b = R.Batch([4], 1, 32, 16)
    with Cache(b, "bf16", cuda_device) as c:
        n = L.lora_kernel_launches()
        e = torch.empty(0, 32, dtype=torch.bfloat16, device=cuda_device)
        none = torch.empty(0, dtype=torch.int32, device=cuda_device)
        L.lora_kv_append(c.kv, 0, e, e.clone(), torch.empty(0, 1, dtype=torch.int32, device=cuda_device), none)
        L.lora_kv_gather(c.kv, 0, e, e.clone(), c.table, c.lens, torch.zeros(2, dtype=torch.int32, device=cuda_device))
        assert L.lora_kernel_launches() == n


def test_refusals(cuda_device):
    b = R.Batch([20, 20], 2, 64, 16, seed=9)
    off, k, v = b.rows()
    k, v, off = k.to(cuda_device), v.to(cuda_device), off.to(cuda_device)
    with Cache(b, "bf16", cuda_device) as c:
        def code(fn=L.lora_kv_append, layer=0, kk=k, vv=v, table=c.table, lens=c.lens, o=off):
            with pytest.raises((L.LoraError, ValueError)) as e:
                fn(c.kv, layer, kk, vv, table, lens, o)
            return getattr(e.value, "code", None)

        n = L.lora_kernel_launches()
        assert code(layer=1) == L.LORA_ERR_INVALID_ARG and code(layer=-1) == L.LORA_ERR_INVALID_ARG
        assert code(o=None) == L.LORA_ERR_INVALID_ARG                      # 40 rows, 2 sequences
        code(kk=k[:, :64]), code(kk=k.float()), code(kk=k.cpu()), code(vv=v[:39])
        code(table=c.table.long()), code(table=c.table[:1]), code(lens=c.lens[:1]), code(o=off[:2])
        wide = torch.zeros(40, 133, dtype=torch.bfloat16, device=cuda_device)
        assert code(kk=wide[:, :128]) == L.LORA_ERR_ALIGNMENT              # a row pitch of 133
        wide = torch.zeros(40, 136, dtype=torch.bfloat16, device=cuda_device)
        assert code(kk=wide[:, 1:129]) == L.LORA_ERR_ALIGNMENT
        assert code(kk=k[:1].expand(40, 128)) == L.LORA_ERR_INVALID_ARG    # rows that share memory
        assert code(fn=L.lora_kv_gather, vv=k) == L.LORA_ERR_INVALID_ARG   # outputs that overlap
        assert L.lora_kernel_launches() == n
        shape = (1, b.n_pages, 16, 2, 64, 0)
        for bad in ((0, 4, 16, 2, 64, 0), (1, 0, 16, 2, 64, 0), (1, 4, 24, 2, 64, 0), (1, 4, 8, 2, 64, 0),
                    (1, 4, 16, 0, 64, 0), (1, 4, 16, 2, 72, 0), (1, 4, 16, 2, 272, 0), (1, 4, 16, 2, 64, 3)):
            assert L.lora_kv_bytes_required(*bad) == 0
            with pytest.raises(L.LoraError):
                L.lora_kv_create(0, *bad, c.mem)
        with pytest.raises(L.LoraError):
            L.lora_kv_create(0, *shape, c.mem[:-1])
        with pytest.raises(L.LoraError):
            L.lora_kv_create(0, *shape, torch.zeros(c.mem.numel() + 256, dtype=torch.uint8, device=cuda_device)[16:])


def test_on_another_stream_and_in_a_graph(cuda_device):
    b = R.Batch([25, 40], 4, 64, 16, seed=10)
    off, k, v = b.rows()
    k, v, off = k.to(cuda_device), v.to(cuda_device), off.to(cuda_device)
    with Cache(b, "e4m3", cuda_device) as c:
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        L.lora_kv_append(c.kv, 0, k, v, c.table, c.lens, off, stream=side)
        L.lora_kv_gather(c.kv, 0, ko, vo, c.table, c.lens, off, stream=side)
        side.synchronize()
        assert same((ko.cpu(), vo.cpu()), c.expect("e4m3"))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lora_kv_append(c.kv, 0, k, v, c.table, c.lens, off)
            L.lora_kv_gather(c.kv, 0, ko, vo, c.table, c.lens, off)
        for seed in (11, 12):  # new values in the same buffers
            n = R.Batch([25, 40], 4, 64, 16, seed=seed)
            c.b.k, c.b.v = n.k, n.v
            _, k2, v2 = n.rows()
            k.copy_(k2), v.copy_(v2)
            graph.replay()
            torch.cuda.synchronize()
            assert same((ko.cpu(), vo.cpu()), c.expect("e4m3"))
