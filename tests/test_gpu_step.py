"""Decode steps of one adapted layer as a serving program runs them:

    residual + norm -> q, k, v (lora_linear) -> lora_kv_append -> lora_attend
    -> o (lora_linear) -> residual + norm

over several steps of a batch that grows, with mixed adapters, a request that
ends and one that joins.  Each stage is compared with its definition on the
stage's own inputs, and a captured step with the calls it captured."""

import numpy as np
import pytest
import torch

import adapter_deltas_b200 as L
import kv_reference as R
import oracle
import synth
from gpu_harness import DevicePool, assert_close, scales_of, to_dev_bf16, to_host_bits

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM, PAGE, EPS = 8, 2, 64, 16, 1e-5
WIDTH, KV_WIDTH = HEADS * DIM, KV_HEADS * DIM
Q, K, V, O = range(4)


class Layer:
    def __init__(self, device, kv_type, T):
        ids = np.array([i % 4 - 1 for i in range(T)], np.int32)  # -1: no adapter
        targets = [(WIDTH, WIDTH), (WIDTH, KV_WIDTH), (WIDTH, KV_WIDTH), (WIDTH, WIDTH)]
        self.w = synth.custom(21, T, targets, [8, 16, 4], 16, ids=ids)
        self.pool = DevicePool(self.w, device)
        self.W = [to_dev_bf16(self.w.W(t), device) for t in range(4)]
        self.ids, self.scales = torch.from_numpy(ids).to(device), torch.from_numpy(scales_of(self.w)).to(device)
        self.ws = torch.empty(max(L.lora_linear_workspace_bytes(self.pool.pool, t, T) for t in range(4)),
                              dtype=torch.uint8, device=device)
        shape = (1, 64, PAGE, KV_HEADS, DIM, R.TYPES[kv_type])
        self.mem = torch.full((L.lora_kv_bytes_required(*shape),), 255, dtype=torch.uint8, device=device)
        self.kv = L.lora_kv_create(device.index, *shape, self.mem)
        self.attend_ws = torch.empty(L.lora_attend_workspace_bytes(self.kv, HEADS), dtype=torch.uint8, device=device)
        g = torch.Generator().manual_seed(5)
        self.norm_w = [(1 + 0.1 * torch.randn(WIDTH, generator=g)).to(torch.bfloat16).to(device) for _ in range(2)]
        self.table = torch.randperm(64, generator=g)[:T * 4].view(T, 4).to(torch.int32).to(device)
        self.lens = torch.zeros(T, dtype=torch.int32, device=device)
        e = lambda n: torch.zeros(T, n, dtype=torch.bfloat16, device=device)  # noqa: E731
        self.x, self.res, self.h, self.qkv, self.att, self.o, self.res2, self.h2 = (
            e(n) for n in (WIDTH, WIDTH, WIDTH, WIDTH + 2 * KV_WIDTH, WIDTH, WIDTH, WIDTH, WIDTH))
        self.h2q = torch.zeros(T, WIDTH, dtype=torch.float8_e4m3fn, device=device)
        self.h2s = torch.zeros(T, WIDTH // 128, device=device)

    def linear(self, target, x, y):
        L.lora_linear(self.pool.pool, target, x, self.W[target], y, self.ids, self.scales, self.ws)

    def parts(self):
        return (self.qkv[:, :WIDTH], self.qkv[:, WIDTH:WIDTH + KV_WIDTH], self.qkv[:, WIDTH + KV_WIDTH:])

    def step(self):
        q, k, v = self.parts()
        L.lora_rmsnorm(self.x, self.norm_w[0], EPS, residual=self.res, residual_out=self.res2, y=self.h)
        for target, y in ((Q, q), (K, k), (V, v)):
            self.linear(target, self.h, y)
        L.lora_kv_append(self.kv, 0, k, v, self.table, self.lens)
        L.lora_attend(self.kv, 0, q, self.att, self.table, self.lens, self.attend_ws)
        self.linear(O, self.att, self.o)
        L.lora_rmsnorm(self.o, self.norm_w[1], EPS, residual=self.res2, residual_out=self.res2, y=self.h2, q=self.h2q,
                       q_scales=self.h2s)

    def close(self):
        L.lora_kv_destroy(self.kv)
        self.pool.close()


def near(got, want, half=R.U_BF16):
    assert ((got.cpu().double() - want).abs() <= want.abs() * (half + 2.0 ** -18)).all()


def check_linear(layer, target, x, y):
    w, ids = layer.w, layer.w.ids
    adapters = {s: w.adapter(s, target) for s in range(w.n_slots)}
    ref, bad = oracle.lora_linear(to_host_bits(x), w.W(target), ids, w.n_slots, adapters, w.alpha)
    assert bad == 0
    assert_close(to_host_bits(y), ref, what="target %d" % target)


@pytest.mark.parametrize("kv_type", list(R.TYPES))
def test_decode_steps(cuda_device, kv_type):
    T, steps = 6, 21  # past a page's end
    layer = Layer(cuda_device, kv_type, T)
    seen_k, seen_v = [[] for _ in range(T)], [[] for _ in range(T)]
    g = torch.Generator().manual_seed(8)
    try:
        lens = [0] * T
        for step in range(steps):
            for i in range(T):
                if i == 2 and step == 9:      # this request ends
                    lens[i] = -1
                elif i == 4 and step < 5:     # this one joins later
                    lens[i] = -1
                elif i == 4 and step == 5:
                    lens[i] = 1
                elif lens[i] >= 0:
                    lens[i] += 1
            layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            layer.x.copy_(torch.randn(T, WIDTH, generator=g).to(torch.bfloat16))
            layer.res.copy_((2 * torch.randn(T, WIDTH, generator=g)).to(torch.bfloat16))
            layer.att.fill_(0.5)
            layer.step()
            torch.cuda.synchronize()
            assert L.lora_get_error(layer.pool.pool) == L.LORA_OK and L.lora_kv_get_error(layer.kv) == L.LORA_OK
            q, k, v = (t.cpu() for t in layer.parts())
            for i, n in enumerate(lens):
                if n > 0:
                    seen_k[i].append(k[i].view(KV_HEADS, DIM)), seen_v[i].append(v[i].view(KV_HEADS, DIM))
            if step not in (0, 6, 15, 16, 20):
                continue
            h, n = R.norm(layer.x.cpu(), layer.res.cpu(), layer.norm_w[0].cpu(), EPS)
            near(layer.h, n)
            for target, y in zip((Q, K, V), layer.parts()):
                check_linear(layer, target, layer.h, y.contiguous())
            for i, count in enumerate(lens):
                if count < 0:
                    assert (layer.att[i] == 0.5).all()
                    continue
                o, _, tol, _ = R.attend(q[i].view(HEADS, DIM), torch.stack(seen_k[i]), torch.stack(seen_v[i]), kv_type,
                                        DIM ** -0.5)
                assert ((layer.att[i].cpu().view(HEADS, DIM).double() - o).abs() <= tol).all()
            check_linear(layer, O, layer.att, layer.o)
            # the second norm's residual is the first one's sum, rounded, updated in place
            h2, n2 = R.norm(layer.o.cpu(), h.float().to(torch.bfloat16), layer.norm_w[1].cpu(), EPS)
            near(layer.res2, h2)
            near(layer.h2, n2)
    finally:
        layer.close()


def test_a_captured_step_replays_the_calls(cuda_device):
    T = 6
    layer = Layer(cuda_device, "e4m3", T)
    g = torch.Generator().manual_seed(9)
    try:
        layer.lens.fill_(1)
        layer.step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.step()
        for lens in ([2, 2, 2, 2, 2, 2], [3, -1, 3, 3, 3, 0], [4, 2, 4, -1, 4, 1]):
            layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            layer.x.copy_(torch.randn(T, WIDTH, generator=g).to(torch.bfloat16))
            layer.res.copy_(torch.randn(T, WIDTH, generator=g).to(torch.bfloat16))
            layer.att.fill_(0.5)
            before = layer.mem.clone()
            layer.step()
            torch.cuda.synchronize()
            want = [t.clone() for t in (layer.att, layer.h2, layer.h2q.view(torch.uint8), layer.h2s, layer.mem)]
            layer.mem.copy_(before)
            layer.att.fill_(0.5)
            graph.replay()
            torch.cuda.synchronize()
            got = (layer.att, layer.h2, layer.h2q.view(torch.uint8), layer.h2s, layer.mem)
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    finally:
        layer.close()
