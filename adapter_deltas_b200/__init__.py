"""Thin Python binding of the B200 multi-LoRA delta library (liblora_b200.so).

Every function here has the name of the C entry point it calls (see
``include/lora.h``) and only marshals arguments: torch tensors become device
pointers, the current CUDA stream becomes the stream argument, and a non-zero
status raises ``LoraError``.  All arithmetic runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback: importing this package fails if
the library has not been built (``python adapter_deltas_b200/_build.py``).

Tensors: x and y are bf16 [T, ld] (row-major, ld >= d and a multiple of 8),
ids int32 [T], scales fp32 [n_slots], workspace uint8; all on the pool's device.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
# LORA_B200_DEBUG=1 selects the bounds-checking build (LORA_DEBUG)
DEBUG_BUILD = os.environ.get("LORA_B200_DEBUG") == "1"
LIB_PATH = os.path.join(_HERE, "liblora_b200_debug.so" if DEBUG_BUILD else "liblora_b200.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "%s is not built; run `python adapter_deltas_b200/_build.py%s` "
        "(the delta path has no fallback)" % (os.path.basename(LIB_PATH), " --debug" if DEBUG_BUILD else ""))

_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t

LORA_OK = 0
LORA_ERR_INVALID_ARG = 1
LORA_ERR_ALIGNMENT = 2
LORA_ERR_NO_PAGES = 3
LORA_ERR_SLOT = 4
LORA_ERR_NOT_LOADED = 5
LORA_ERR_CUDA = 6
LORA_ERR_BAD_ID = 7
LORA_ERR_TIMEOUT = 8
LORA_ERR_WORKSPACE = 9
LORA_ERR_BOUNDS = 10

LORA_KV_BF16 = 0
LORA_KV_E4M3 = 1
LORA_KV_INT8 = 2


class lora_target(ctypes.Structure):
    _fields_ = [("d_in", _I), ("d_out", _I)]


class lora_pool_info(ctypes.Structure):
    _fields_ = [("slot_bytes", _Z), ("page_bytes", _Z), ("pages_per_slot", _I), ("n_pages", _I),
                ("free_pages", _I), ("n_slots", _I), ("n_targets", _I), ("r_max", _I),
                ("decode_ctas", _I)]


class lora_plan_layout(ctypes.Structure):
    _fields_ = [("header", _Z), ("perm", _Z), ("seg_start", _Z), ("seg_slot", _Z), ("items", _Z),
                ("tiles", _Z), ("total", _Z), ("s_max", _I), ("i_max", _I), ("j_max", _I)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_sig("lora_status_string", ctypes.c_char_p, [_I])
_sig("lora_pool_bytes_required", _Z, [_P, _I, _I, _I, _Z])
_sig("lora_pool_create", _I, [ctypes.POINTER(_P), _I, _P, _I, _I, _I, _Z, _P, _Z, ctypes.c_uint64])
_sig("lora_pool_load", _I, [_P, _I, _I, _I, _P, _P, _I, _P])
_sig("lora_pool_unload", _I, [_P, _I])
_sig("lora_pool_swap_in", _I, [_P, _I, _P, _P, _Z, _P, _Z, _P])
_sig("lora_swap_src_bytes", _Z, [_P, _P])
_sig("lora_swap_staging_bytes", _Z, [_P, _P])
_sig("lora_pool_destroy", _I, [_P])
_sig("lora_pool_page_table", _P, [_P])
_sig("lora_pool_get_info", _I, [_P, ctypes.POINTER(lora_pool_info)])
_sig("lora_pool_target_offsets", _I, [_P, _I, ctypes.POINTER(_Z), ctypes.POINTER(_Z)])
_sig("lora_workspace_bytes", _Z, [_P, _I, _I])
_sig("lora_linear_workspace_bytes", _Z, [_P, _I, _I])
_sig("lora_plan_layout_get", _I, [_P, _I, ctypes.POINTER(lora_plan_layout)])
_sig("lora_plan_ids", _I, [_P, _P, _I, _P, _Z, _P])
_sig("lora_plan_segments", _I, [_P, _P, _P, _I, _I, _P, _Z, _P])
_sig("lora_mma_min_rows", _I, [])
_sig("lora_mma_min_rows_for", _I, [_I, _I])
_sig("lora_apply_plan", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _Z, _P])
_sig("lora_apply", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _P, _Z, _P])
_sig("lora_apply_segments", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _P, _Z, _P])
_sig("lora_apply_multi", _I, [_P, _I, _P, _P, _I, _P, _I, _P, _P, _P, _I, _P, _Z, _P])
_sig("lora_linear", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _P, _I, _P, _Z, _P])
_sig("lora_linear_expand", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _P, _I, _P])
_sig("lora_apply_moe", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _I, _I, _P, _P, _Z, _P])
_sig("lora_moe_workspace_bytes", _Z, [_P, _I, _I])
_sig("lora_shrink", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _Z, _P])
_sig("lora_expand", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _P, _Z, _P])
_sig("lora_apply_noalloc", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _P])
_sig("lora_kv_bytes_required", _Z, [_I, _I, _I, _I, _I, _I])
_sig("lora_kv_create", _I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _I, _I, _P, _Z])
_sig("lora_kv_destroy", _I, [_P])
_sig("lora_kv_get_error", _I, [_P, ctypes.POINTER(_I), _P])
_sig("lora_kv_append", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _P, _I, _I, _P])
_sig("lora_kv_gather", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _P, _I, _I, _P])
_sig("lora_attend_workspace_bytes", _Z, [_P, _I])
_sig("lora_attend", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _P, _I, ctypes.c_float, _I, _P, _Z, _P])
_sig("lora_selftest_stalled_attend", _I, [_P, _I, _P, _I, _P, _I, _I, _P, _I, _P, _I, _P, _Z, _P])
_sig("lora_selftest_late_lane_attend", _I, [_P, _I, _P, _I, _P, _I, _I, _P, _I, _P, _I, _P, _Z, _I, _P])
_sig("lora_rmsnorm", _I, [_I, _P, _I, _P, _I, _P, _I, _P, ctypes.c_float, _P, _I, _P, _I, _P, _I, _I, _I, _P])
_sig("lora_get_error", _I, [_P, ctypes.POINTER(_I), _P])
_sig("lora_kernel_launches", ctypes.c_uint64, [])
_sig("lora_set_wait_limit_ns", None, [ctypes.c_uint64])
_sig("lora_selftest_stalled_apply", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _P])


class LoraError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s failed: %s" % (where, lora_status_string(code)))


def _check(code: int, where: str) -> None:
    if code != LORA_OK:
        raise LoraError(code, where)


def lora_status_string(code: int) -> str:
    return _lib.lora_status_string(code).decode()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ld(t) -> int:
    return int(t.stride(0)) if t is not None and t.dim() == 2 else 0


def _targets(targets: Sequence[Tuple[int, int]]):
    arr = (lora_target * len(targets))()
    for i, (d_in, d_out) in enumerate(targets):
        arr[i].d_in = int(d_in)
        arr[i].d_out = int(d_out)
    return arr


class PoolHandle:
    """The opaque pool pointer plus the Python objects it must outlive."""

    def __init__(self, ptr: int, device: int, mem, targets, r_max: int, n_slots: int):
        self.ptr = ptr
        self.device = device
        self.mem = mem
        self.targets = list(targets)
        self.r_max = r_max
        self.n_slots = n_slots

    @property
    def _as_parameter_(self):
        return self.ptr


# ---------------------------------------------------------------- pool


def lora_pool_bytes_required(targets, r_max: int, n_slots: int, page_bytes: int = 0) -> int:
    arr = _targets(targets)
    return int(_lib.lora_pool_bytes_required(arr, len(arr), r_max, n_slots, page_bytes))


def lora_pool_create(device: int, targets, r_max: int, n_slots: int, page_bytes: int, pool_mem,
                     scatter_seed: int = 0) -> PoolHandle:
    arr = _targets(targets)
    out = _P()
    nbytes = pool_mem.numel() * pool_mem.element_size()
    _check(_lib.lora_pool_create(ctypes.byref(out), device, arr, len(arr), r_max, n_slots, page_bytes,
                                 _ptr(pool_mem), nbytes, scatter_seed), "lora_pool_create")
    return PoolHandle(out.value, device, pool_mem, targets, r_max, n_slots)


def lora_pool_load(pool: PoolHandle, slot: int, target: int, rank: int, A, B, stream=None) -> None:
    """A: bf16 [rank, d_in], B: bf16 [d_out, rank]; torch tensors on the pool's
    device or on the host (contiguous)."""
    on_dev = 1 if (A is not None and A.is_cuda) else 0
    if A is not None:
        assert A.is_contiguous() and B.is_contiguous()
    _check(_lib.lora_pool_load(pool, slot, target, rank, _ptr(A), _ptr(B), on_dev, _stream(stream)),
           "lora_pool_load")


def _int_array(values):
    values = [int(v) for v in values]
    return (ctypes.c_int * len(values))(*values)


def lora_swap_src_bytes(pool: PoolHandle, ranks) -> int:
    return int(_lib.lora_swap_src_bytes(pool, _int_array(ranks)))


def lora_swap_staging_bytes(pool: PoolHandle, ranks) -> int:
    return int(_lib.lora_swap_staging_bytes(pool, _int_array(ranks)))


def lora_pool_swap_in(pool: PoolHandle, slot: int, ranks, src, staging, stream=None) -> None:
    """One adapter, all targets, from host memory `src` (a CPU tensor, pinned
    for an asynchronous copy) through the device tensor `staging`."""
    nbytes = src.numel() * src.element_size()
    _check(_lib.lora_pool_swap_in(pool, slot, _int_array(ranks), _ptr(src), nbytes, _ptr(staging),
                                  staging.numel() * staging.element_size(), _stream(stream)), "lora_pool_swap_in")


def lora_pool_unload(pool: PoolHandle, slot: int) -> None:
    _check(_lib.lora_pool_unload(pool, slot), "lora_pool_unload")


def lora_pool_destroy(pool: PoolHandle) -> None:
    if pool.ptr:
        _check(_lib.lora_pool_destroy(pool), "lora_pool_destroy")
        pool.ptr = 0


def lora_pool_page_table(pool: PoolHandle) -> int:
    return int(_lib.lora_pool_page_table(pool) or 0)


def lora_pool_get_info(pool: PoolHandle) -> lora_pool_info:
    info = lora_pool_info()
    _check(_lib.lora_pool_get_info(pool, ctypes.byref(info)), "lora_pool_get_info")
    return info


def lora_pool_target_offsets(pool: PoolHandle, target: int) -> Tuple[int, int]:
    a, b = _Z(), _Z()
    _check(_lib.lora_pool_target_offsets(pool, target, ctypes.byref(a), ctypes.byref(b)),
           "lora_pool_target_offsets")
    return int(a.value), int(b.value)


# ---------------------------------------------------------------- plans


def lora_workspace_bytes(pool: PoolHandle, target: int, max_tokens: int) -> int:
    return int(_lib.lora_workspace_bytes(pool, target, max_tokens))


def lora_plan_layout_get(pool: PoolHandle, T: int) -> lora_plan_layout:
    out = lora_plan_layout()
    _check(_lib.lora_plan_layout_get(pool, T, ctypes.byref(out)), "lora_plan_layout_get")
    return out


def lora_mma_min_rows() -> int:
    return int(_lib.lora_mma_min_rows())


def lora_mma_min_rows_for(n_segments: int, T: int) -> int:
    """Segment length from which a segment plan of this batch uses the tensor cores."""
    return int(_lib.lora_mma_min_rows_for(n_segments, T))


def lora_plan_ids(pool: PoolHandle, ids, ws, stream=None) -> None:
    _check(_lib.lora_plan_ids(pool, _ptr(ids), ids.shape[0], _ptr(ws), ws.numel(), _stream(stream)),
           "lora_plan_ids")


def lora_plan_segments(pool: PoolHandle, seg_offsets, seg_slot, T: int, ws, stream=None) -> None:
    _check(_lib.lora_plan_segments(pool, _ptr(seg_offsets), _ptr(seg_slot), seg_slot.shape[0], T, _ptr(ws),
                                   ws.numel(), _stream(stream)), "lora_plan_segments")


# ---------------------------------------------------------------- compute


def lora_apply_plan(pool: PoolHandle, target: int, x, y, scales, ws, stream=None) -> None:
    _check(_lib.lora_apply_plan(pool, target, _ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(scales), y.shape[0],
                                _ptr(ws), ws.numel(), _stream(stream)), "lora_apply_plan")


def lora_apply(pool: PoolHandle, target: int, x, y, ids, scales, ws, stream=None) -> None:
    _check(_lib.lora_apply(pool, target, _ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(ids), _ptr(scales),
                           y.shape[0], _ptr(ws), ws.numel(), _stream(stream)), "lora_apply")


def lora_apply_multi(pool: PoolHandle, targets, x, y, y_cols, ids, scales, ws, stream=None) -> None:
    """Several same-shape targets sharing x in one call; target i adds its
    delta to columns y_cols[i] .. y_cols[i] + d_out - 1 of y."""
    n = len(targets)
    t_arr = (ctypes.c_int * n)(*[int(t) for t in targets])
    c_arr = (ctypes.c_int * n)(*[int(c) for c in y_cols])
    _check(_lib.lora_apply_multi(pool, n, t_arr, _ptr(x), _ld(x), _ptr(y), _ld(y), c_arr, _ptr(ids), _ptr(scales),
                                 y.shape[0], _ptr(ws), ws.numel(), _stream(stream)), "lora_apply_multi")


def lora_apply_segments(pool: PoolHandle, target: int, x, y, seg_offsets, seg_slot, scales, ws,
                        stream=None) -> None:
    _check(_lib.lora_apply_segments(pool, target, _ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(seg_offsets),
                                    _ptr(seg_slot), seg_slot.shape[0], _ptr(scales), y.shape[0], _ptr(ws),
                                    ws.numel(), _stream(stream)), "lora_apply_segments")


def lora_linear_workspace_bytes(pool: PoolHandle, target: int, max_tokens: int) -> int:
    return int(_lib.lora_linear_workspace_bytes(pool, target, max_tokens))


def lora_linear(pool: PoolHandle, target: int, x, W, y, ids, scales, ws, stream=None) -> None:
    """y = x W^T + each row's delta, written once (W: [d_out, d_in] row-major)."""
    _check(_lib.lora_linear(pool, target, _ptr(x), _ld(x), _ptr(W), _ld(W), _ptr(y), _ld(y), _ptr(ids),
                            _ptr(scales), y.shape[0], _ptr(ws), ws.numel(), _stream(stream)), "lora_linear")


def lora_linear_expand(pool: PoolHandle, target: int, x, W, v, y, ids, scales, stream=None) -> None:
    """y = x W^T + each row's s_a B_a v[t] (v from lora_shrink), written once."""
    _check(_lib.lora_linear_expand(pool, target, _ptr(x), _ld(x), _ptr(W), _ld(W), _ptr(v), _ld(v), _ptr(y),
                                   _ld(y), _ptr(ids), _ptr(scales), y.shape[0], _stream(stream)),
           "lora_linear_expand")


def lora_moe_workspace_bytes(pool: PoolHandle, target: int, max_pairs: int) -> int:
    return int(_lib.lora_moe_workspace_bytes(pool, target, max_pairs))


def lora_apply_moe(pool: PoolHandle, target: int, x, y, lora_ids, topk_ids, n_experts: int, scales, ws,
                   stream=None) -> None:
    """Routed expert pairs: y[t * k + j] += s B_s (A_s x[t]), s = lora_ids[t] * n_experts + topk_ids[t, j];
    x [T, d_in], y [T * k, d_out], topk_ids [T, k]."""
    T, k = int(topk_ids.shape[0]), int(topk_ids.shape[1])
    _check(_lib.lora_apply_moe(pool, target, _ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(lora_ids), _ptr(topk_ids), T,
                               k, n_experts, _ptr(scales), _ptr(ws), ws.numel(), _stream(stream)),
           "lora_apply_moe")


def lora_shrink(pool: PoolHandle, target: int, x, ids, v, ws, stream=None) -> None:
    _check(_lib.lora_shrink(pool, target, _ptr(x), _ld(x), _ptr(ids), ids.shape[0], _ptr(v), _ld(v), _ptr(ws),
                            ws.numel(), _stream(stream)), "lora_shrink")


def lora_expand(pool: PoolHandle, target: int, v, y, ids, scales, ws, stream=None) -> None:
    _check(_lib.lora_expand(pool, target, _ptr(v), _ld(v), _ptr(y), _ld(y), _ptr(ids), _ptr(scales),
                            ids.shape[0], _ptr(ws), ws.numel(), _stream(stream)), "lora_expand")


LORA_NOALLOC_MAX_TOKENS = 4096


def lora_apply_noalloc(pool: PoolHandle, target: int, x, y, ids, scales, stream=None) -> None:
    """lora_apply without a workspace argument: the workspace lives in a fixed
    device array inside the library (for callers that cannot allocate).
    Calls that overlap on the GPU share that array and must be serialised."""
    _check(_lib.lora_apply_noalloc(pool, target, _ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(ids), _ptr(scales),
                                   y.shape[0], _stream(stream)), "lora_apply_noalloc")


# ---------------------------------------------------------------- the key/value cache


class KvHandle:
    """The opaque cache pointer plus the Python objects it must outlive."""

    def __init__(self, ptr: int, device: int, mem, n_layers: int, n_pages: int, page_tokens: int, n_kv_heads: int,
                 head_dim: int, kv_type: int):
        self.ptr = ptr
        self.device = device
        self.mem = mem
        self.n_layers, self.n_pages, self.page_tokens = n_layers, n_pages, page_tokens
        self.n_kv_heads, self.head_dim, self.kv_type = n_kv_heads, head_dim, kv_type

    @property
    def _as_parameter_(self):
        return self.ptr


# The calls below run once or twice per layer of a step, some of them for a few
# microseconds on the GPU: their checks read each property of a tensor once.


def _refuse_past_int(bits: int, where: str) -> None:
    """bits: sizes and indices or'ed together; one past a C int (which ctypes would cut) or below 0 is refused."""
    if bits >> 31:
        _check(LORA_ERR_INVALID_ARG, where)


def _rows(t, name: str, device: int, shape, dtype, where: str):
    """Address and leading dimension of a [T, ld] operand whose rows of shape[1] values are reached by its row stride."""
    if t.shape == shape and t.is_contiguous() and t.dtype is dtype and t.get_device() == device:
        return t.data_ptr(), shape[1]
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError("%s: %s must be %s %s with unit column stride on cuda:%d, not %s %s %s"
                         % (where, name, dtype, list(shape), device, t.dtype, tuple(t.shape), t.device))
    ld = t.stride(0) if shape[0] > 1 else (shape[1] + 7) // 8 * 8
    _refuse_past_int(ld, where)
    return t.data_ptr(), ld


def _dense(t, name: str, device: int, shape, dtype, where: str) -> int:
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: %s must be contiguous %s %s on cuda:%d, not %s %s %s"
                         % (where, name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _stream_on(stream, device: int) -> int:
    """The stream argument of a call on `device`; the current stream of that device by default."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(device)  # (current_stream() makes an object, about 1 us)
    return stream if isinstance(stream, int) else stream.cuda_stream


def lora_kv_bytes_required(n_layers: int, n_pages: int, page_tokens: int, n_kv_heads: int, head_dim: int,
                           kv_type: int) -> int:
    if (n_layers | n_pages | page_tokens | n_kv_heads | head_dim | kv_type) >> 31:
        return 0
    return int(_lib.lora_kv_bytes_required(n_layers, n_pages, page_tokens, n_kv_heads, head_dim, kv_type))


def lora_kv_create(device: int, n_layers: int, n_pages: int, page_tokens: int, n_kv_heads: int, head_dim: int,
                   kv_type: int, kv_mem) -> KvHandle:
    """A paged key/value cache over the device tensor `kv_mem`."""
    if kv_mem.get_device() != device or not kv_mem.is_contiguous():
        raise ValueError("lora_kv_create: kv_mem must be contiguous on cuda:%d" % device)
    _refuse_past_int(n_layers | n_pages | page_tokens | n_kv_heads | head_dim | kv_type, "lora_kv_create")
    out = _P()
    _check(_lib.lora_kv_create(ctypes.byref(out), device, n_layers, n_pages, page_tokens, n_kv_heads, head_dim, kv_type,
                               kv_mem.data_ptr(), kv_mem.numel() * kv_mem.element_size()), "lora_kv_create")
    return KvHandle(out.value, device, kv_mem, n_layers, n_pages, page_tokens, n_kv_heads, head_dim, kv_type)


def lora_kv_destroy(kv: KvHandle) -> None:
    ptr, kv.ptr = kv.ptr, 0  # (freed even where the call reports an error: not to be passed again)
    if ptr:
        _check(_lib.lora_kv_destroy(ptr), "lora_kv_destroy")


def lora_kv_get_error(kv: KvHandle, stream=None) -> int:
    st = _I(0)
    _check(_lib.lora_kv_get_error(kv, ctypes.byref(st), _stream_on(stream, kv.device)), "lora_kv_get_error")
    return int(st.value)


def _kv_rows(fn, where: str, kv: KvHandle, layer: int, k, v, page_table, seq_lens, row_offsets, stream) -> None:
    import torch
    dev, T, n, paged = kv.device, k.shape[0], seq_lens.shape[0], page_table.shape
    if len(paged) != 2:
        raise ValueError("%s: page_table must be [n_seqs, max_pages]" % where)
    _refuse_past_int(layer | T | n | paged[1], where)
    shape = (T, kv.n_kv_heads * kv.head_dim)
    kp, ldk = _rows(k, "k", dev, shape, torch.bfloat16, where)
    vp, ldv = _rows(v, "v", dev, shape, torch.bfloat16, where)
    table = _dense(page_table, "page_table", dev, (n, paged[1]), torch.int32, where)
    lens = _dense(seq_lens, "seq_lens", dev, (n,), torch.int32, where)
    off = None if row_offsets is None else _dense(row_offsets, "row_offsets", dev, (n + 1,), torch.int32, where)
    _check(fn(kv, layer, kp, ldk, vp, ldv, table, paged[1], lens, off, n, T, _stream_on(stream, dev)), where)


def lora_kv_append(kv: KvHandle, layer: int, k, v, page_table, seq_lens, row_offsets=None, stream=None) -> None:
    """New tokens into the cache: k, v bf16 [T, n_kv_heads * head_dim] (column slices of wider rows will do),
    page_table int32 [n_seqs, max_pages], seq_lens int32 [n_seqs] (these tokens included), row_offsets int32
    [n_seqs + 1] or None for one row per sequence."""
    _kv_rows(_lib.lora_kv_append, "lora_kv_append", kv, layer, k, v, page_table, seq_lens, row_offsets, stream)


def lora_kv_gather(kv: KvHandle, layer: int, k, v, page_table, seq_lens, row_offsets=None, stream=None) -> None:
    """Held tokens back into k, v (bf16): the converse of lora_kv_append."""
    _kv_rows(_lib.lora_kv_gather, "lora_kv_gather", kv, layer, k, v, page_table, seq_lens, row_offsets, stream)


def lora_attend_workspace_bytes(kv: KvHandle, n_heads: int) -> int:
    return 0 if n_heads >> 31 else int(_lib.lora_attend_workspace_bytes(kv, n_heads))


def lora_attend(kv: KvHandle, layer: int, q, out, page_table, seq_lens, ws, scale: Optional[float] = None,
                window: int = 0, sinks=None, lse=None, stream=None) -> None:
    """Attention of one new token per sequence over the cache: q, out bf16 [n_seqs, n_heads * head_dim]; scale
    1 / sqrt(head_dim) by default; sinks fp32 [n_heads] or None; lse fp32 [n_seqs, n_heads] or None.  A window past
    2^30 is all of any sequence."""
    import torch
    dev, n, width, paged = kv.device, seq_lens.shape[0], q.shape[-1], page_table.shape
    where, n_heads = "lora_attend", width // kv.head_dim
    if width % kv.head_dim or len(paged) != 2:
        raise ValueError("%s: q must be [n_seqs, n_heads * head_dim], page_table [n_seqs, max_pages]" % where)
    _refuse_past_int(layer | n | paged[1] | n_heads | (-1 if window < 0 else 0), where)
    shape = (n, width)
    qp, ldq = _rows(q, "q", dev, shape, torch.bfloat16, where)
    op, ldo = _rows(out, "out", dev, shape, torch.bfloat16, where)
    table = _dense(page_table, "page_table", dev, (n, paged[1]), torch.int32, where)
    lens = _dense(seq_lens, "seq_lens", dev, (n,), torch.int32, where)
    sp = None if sinks is None else _dense(sinks, "sinks", dev, (n_heads,), torch.float32, where)
    lp = None if lse is None else _dense(lse, "lse", dev, (n, n_heads), torch.float32, where)
    ws_bytes = ws.numel()
    wp = _dense(ws, "ws", dev, (ws_bytes,), torch.uint8, where)
    _check(_lib.lora_attend(kv, layer, qp, ldq, op, ldo, lp, sp, n_heads, table, paged[1], lens, n,
                            kv.head_dim ** -0.5 if scale is None else scale, min(window, 1 << 30), wp,
                            ws_bytes, _stream_on(stream, dev)), where)


def lora_rmsnorm(x, weight, eps: float, residual=None, residual_out=None, y=None, q=None, q_scales=None,
                 stream=None) -> None:
    """h = x + residual and its root-mean-square norm: h to residual_out, the norm to y (bf16) and / or q
    (float8_e4m3fn) with q_scales fp32 [T] (one per row) or [T, d / group]."""
    import torch
    where, dev, shape, bf16 = "lora_rmsnorm", x.get_device(), x.shape, torch.bfloat16
    T, d = shape
    _refuse_past_int(T | d, where)
    xp, ldx = _rows(x, "x", dev, shape, bf16, where)
    wp = _dense(weight, "weight", dev, (d,), bf16, where)
    rp = op = yp = qp = None
    ldr = ldo = ldy = ldq = 0
    if residual is not None:
        rp, ldr = _rows(residual, "residual", dev, shape, bf16, where)
    if residual_out is not None:
        op, ldo = _rows(residual_out, "residual_out", dev, shape, bf16, where)
    if y is not None:
        yp, ldy = _rows(y, "y", dev, shape, bf16, where)
    if q is not None:
        qp, ldq = _rows(q, "q", dev, shape, torch.float8_e4m3fn, where)
    group, sp = 0, None
    if q is not None:
        if q_scales is None:
            raise ValueError("%s: q needs q_scales" % where)
        grid = q_scales.shape
        if len(grid) == 2:
            n = grid[1]
            if n < 1 or d % n:
                raise ValueError("%s: q_scales must be [T] or [T, d / group]" % where)
            group = d // n if n > 1 else 0
            sp = _dense(q_scales, "q_scales", dev, (T, n), torch.float32, where)
        else:
            sp = _dense(q_scales, "q_scales", dev, (T,), torch.float32, where)
    _check(_lib.lora_rmsnorm(dev, xp, ldx, rp, ldr, op, ldo, wp, eps, yp, ldy, qp, ldq, sp, group, T, d,
                             _stream_on(stream, dev)), where)


def lora_get_error(pool: PoolHandle, stream=None) -> int:
    st = _I(0)
    _check(_lib.lora_get_error(pool, ctypes.byref(st), _stream(stream)), "lora_get_error")
    return int(st.value)


def lora_kernel_launches() -> int:
    return int(_lib.lora_kernel_launches())


def lora_set_wait_limit_ns(ns: int) -> None:
    """Wall-clock limit of the decode and attention kernels' bounded waits (0: one second)."""
    _lib.lora_set_wait_limit_ns(int(ns))


def lora_selftest_stalled_apply(pool: PoolHandle, target: int, x, y, ids, scales, stream=None) -> None:
    """Test only: the decode launch of lora_apply with no stage ever filled,
    so that its waits run out (LORA_ERR_TIMEOUT in the sticky status)."""
    _check(_lib.lora_selftest_stalled_apply(pool, target, _ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(ids),
                                            _ptr(scales), y.shape[0], _stream(stream)),
           "lora_selftest_stalled_apply")


def lora_selftest_stalled_attend(kv: KvHandle, layer: int, q, out, page_table, seq_lens, ws, stream=None) -> None:
    """Test only: lora_attend with nothing fetched, so that its waits run out
    (LORA_ERR_TIMEOUT in the cache's sticky status)."""
    _check(_lib.lora_selftest_stalled_attend(kv, layer, q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0),
                                             q.shape[1] // kv.head_dim, page_table.data_ptr(), page_table.shape[1],
                                             seq_lens.data_ptr(), seq_lens.shape[0], ws.data_ptr(), ws.numel(),
                                             _stream_on(stream, kv.device)), "lora_selftest_stalled_attend")


def lora_selftest_late_lane_attend(kv: KvHandle, layer: int, q, out, page_table, seq_lens, ws, lane: int, stream=None) -> None:
    """Test only: lora_attend (scale 1) whose warps' lane `lane` finds its waits run out
    from the third step on (LORA_ERR_TIMEOUT in the cache's sticky status)."""
    _check(_lib.lora_selftest_late_lane_attend(kv, layer, q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0),
                                               q.shape[1] // kv.head_dim, page_table.data_ptr(), page_table.shape[1],
                                               seq_lens.data_ptr(), seq_lens.shape[0], ws.data_ptr(), ws.numel(), lane,
                                               _stream_on(stream, kv.device)), "lora_selftest_late_lane_attend")
