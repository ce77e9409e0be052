// kv.cu -- the paged key/value cache: handle, quantising append, read-back.
//
// The cache lives in pages of caller-owned memory located through a page table,
// the unified paging of "Multi-LoRA Serving: Sharing One GPU Across Adapters"
// (section "How S-LoRA Proved the Model") for the other half of what a serving
// GPU holds.  append writes new keys and values (held as bf16, e4m3 or int8,
// kv.cuh), gather reads held rows back as bf16.  Both are one pass over their
// bytes; what bounds them is HBM.
//
// Work split: a row of one head's K or V (a vector) is handled by `lanes`
// neighbouring threads (a power of two), each with 16 bytes of the held row: 8
// elements of bf16 or 16 in 8 bits, whose largest magnitude they reduce with
// shuffles.  An append's block takes `rows` consecutive rows of the batch, so
// many that the blocks are resident at once: its start, a chain of dependent
// reads, is paid once, beside its first loads (4096 rows of 32 heads of 128 as
// e4m3: 25 us, 102 MB at 4.0 TB/s; int8 30; bf16 26.5, 134 MB at 5.1; with 1 row a
// block e4m3 29).  The 8-bit append is bound by neither (issue slots 67 % in use, DRAM
// 33 %): its loads, the maximum over a vector's threads and the quotients follow
// one another.  Addresses are kept per thread and stepped.  A gather's block takes what its threads hold in flight
// twice over: its accesses, 128 bytes of a head here and there, are then close in
// time to the rest of their tiles (11734 rows of that cache: 50 us, 291 MB at
// 5.8 TB/s, int8 51; bf16 64, 385 MB at 6.0; resident blocks of 16 rows 60, 1 row,
// which leaves threads idle, 63).
// The block's warps look up the rows' sequences (a 32-way search in
// row_offsets, two dependent reads up to 1024 sequences, where the row before is
// not in the same one), then a thread a row its length and page; append reads
// its first input rows, which do not depend on that, before.
#include <new>

#include "kv.cuh"

namespace lora {

constexpr int kRowThreads = 256, kRowBlocks = 5;  // blocks resident on an SM
constexpr int kMaxBlockRows = 64;
constexpr int kGatherAhead = 4;  // vectors of a thread in flight
constexpr int kGatherTurns = 2;

// Sequence of row t (largest s with off[s] <= t, if t < off[s + 1]), by one warp; -1 if none.
__device__ __forceinline__ int find_seq(const int32_t *off, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = (hi - lo) / 32 + 1;
    const int i = lo + lane * step;
    const unsigned below = __ballot_sync(~0u, i <= hi && __ldg(off + i) <= t);
    const int c = __popc(below);
    if (c == 0) return -1;
    hi = min(hi, lo + c * step - 1);
    lo += (c - 1) * step;
    if (lo > hi) return -1;  // (offsets out of order)
    if (step == 1) break;
  }
  if (lo >= n) return -1;
  return __ldg(off + lo) <= t && t < __ldg(off + lo + 1) ? lo : -1;
}

// Where rows first .. first + rows - 1 of the batch live: tile[i] = byte offset
// of the tile of head 0, or -1 (not held); tok[i] = the token's row in it.
__device__ __forceinline__ void locate_rows(const KvView &kv, const KvSeqs &s, int first, int rows, long long *tile,
                                            int *tok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (s.offsets) {
    int seq = -1, from = 0, to = 0;
    for (int i = warp; i < rows; i += kRowThreads / 32) {
      const int t = first + i;
      if (t < from || t >= to) {
        seq = find_seq(s.offsets, s.n, t);
        from = to = 0;
        if (seq >= 0) {
          from = __ldg(s.offsets + seq);
          to = __ldg(s.offsets + seq + 1);
        }
      }
      if (lane == 0) {
        tile[i] = seq >= 0 ? (long long)from << 32 | (unsigned)to : 0;
        tok[i] = seq;
      }
    }
    __syncthreads();
  }
  const int i = threadIdx.x;
  if (i < rows) {
    const int t = first + i;
    int seq = t, back = 1;  // the row's distance from its sequence's end
    long long own = 1;      // the sequence's rows (of offsets in error more than 32 bits hold)
    if (s.offsets) {
      seq = tok[i];
      back = (int)tile[i] - t;
      own = (long long)(int)tile[i] - (tile[i] >> 32);
    }
    long long at = -1;
    int row = 0;
    if (seq >= 0) {
      const int len = s.lens[seq];
      const bool none = len == -1 || (len == 0 && !s.offsets);
      if (!none) {
        if (len > 0 && kv_len_ok(kv, s, len) && own <= len) {
          const int pos = len - back;
          at = kv_tile_offset(kv, s.table[(long long)seq * s.max_pages + (pos >> kv.log2_page)], pos);
          row = pos & (kTileTokens - 1);
        }
        if (at < 0) set_status(kv.status, LORA_ERR_BAD_ID);
      }
    }
    tile[i] = at;
    tok[i] = row;
  }
}

// row_offsets must not decrease and stay inside [0, T]; each block checks a share.
__device__ __forceinline__ void check_offsets(const KvView &kv, const KvSeqs &s, int T) {
  if (!s.offsets) return;
  for (int i = blockIdx.x * kRowThreads + threadIdx.x; i <= s.n; i += gridDim.x * kRowThreads) {
    const int a = __ldg(s.offsets + i);
    if (a < 0 || a > T || (i < s.n && __ldg(s.offsets + i + 1) < a)) set_status(kv.status, LORA_ERR_BAD_ID);
  }
}

struct RowArgs {
  uint8_t *k, *v;     // [T, ld] bf16: read (append) or written (gather)
  long long ldk, ldv; // bytes
  int T, rows;        // rows per block
  int lanes;          // threads per vector (power of two >= dim / vec_elements)
  int wide;           // rows start at multiples of 32 bytes
};
__host__ __device__ constexpr int vec_elements(int type) { return 16 / kv_elt(type); }  // of a thread: 16 held bytes

// A thread's 16 values of a bf16 row are 32 bytes.  As one access they are a sector
// of its own; in two halves every sector is touched twice (gather of 11734 rows of
// 32 heads of 128, e4m3: 50 and 54 us).
__device__ __forceinline__ void load32(const uint8_t *p, bool wide, uint4 &a, uint4 &b) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = __ldg(reinterpret_cast<const uint4 *>(p));
    b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  }
}
__device__ __forceinline__ void store32(uint8_t *p, bool wide, const uint4 &a, const uint4 &b) {
  if (wide) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    __stcs(reinterpret_cast<uint4 *>(p), a);
    __stcs(reinterpret_cast<uint4 *>(p) + 1, b);
  }
}

// The vectors of a block are numbered (row, K or V, head), heads fastest, as the
// rows lie in memory; a thread takes every `step`-th.
struct RowWalk {
  int head, x;           // x = 2 * row + which
  int by_head, by_x;     // step, as heads and x
  __device__ RowWalk(int w, int step, int heads) {
    x = w / heads;
    head = w - x * heads;
    by_x = step / heads;
    by_head = step - by_x * heads;
  }
  __device__ void next(int heads) {
    head += by_head;
    x += by_x;
    if (head >= heads) {
      head -= heads;
      ++x;
    }
  }
};

// A thread's place in the held rows: the 16-byte chunk that starts with element e of a vector.
template <int TYPE>
struct HeldPlace {
  int chunk;         // its bytes from the row's start
  int shift, mask;   // of kv_chunk: chunk ^ (token >> shift & mask)
  int row_bytes, head_stride;  // (a page is under 2 GiB)
  __device__ HeldPlace(const KvView &kv, int e) {
    row_bytes = kv.dim * kv_elt(TYPE);
    const int low = (row_bytes / 16) & -(row_bytes / 16);
    chunk = e * kv_elt(TYPE);
    mask = min(low, 8) - 1;
    shift = 3 - __popc(mask);
    head_stride = (int)kv_head_stride(kv);
  }
  __device__ uint4 *operator()(uint8_t *tile, int tok, int which, int head) const {
    return reinterpret_cast<uint4 *>(tile + head * head_stride + (which * kTileTokens + tok) * row_bytes +
                                     (chunk ^ (tok >> shift & mask) << 4));
  }
  __device__ float *scale(uint8_t *tile, int tok, int which, int head) const {
    return reinterpret_cast<float *>(tile + head * head_stride + 2 * kTileTokens * row_bytes) + which * kTileTokens + tok;
  }
};

template <int TYPE>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks) kv_append_kernel(KvView kv, KvSeqs s, RowArgs a) {
  constexpr int E = vec_elements(TYPE), U = E / 8, kAhead = 4 / U;
  __shared__ long long tile[kMaxBlockRows];
  __shared__ int tok[kMaxBlockRows];
  const int first = blockIdx.x * a.rows, rows = min(a.rows, a.T - first);
  const int part = threadIdx.x & (a.lanes - 1), e = part * E, step = kRowThreads / a.lanes;
  const bool on = e < kv.dim;
  const HeldPlace<TYPE> held(kv, e);
  const uint8_t *src_k = a.k + first * a.ldk + e * 2, *src_v = a.v + first * a.ldv + e * 2;
  RowWalk in(threadIdx.x / a.lanes, step, kv.heads), to = in;
  const int turns = (rows * 2 * kv.heads + step * kAhead - 1) / (step * kAhead);
  griddep_wait();
  griddep_launch_dependents();
  for (int turn = 0; turn < turns; ++turn) {  // (every thread takes every turn: the shuffles are the whole warp's)
    uint4 u[kAhead][U];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
#pragma unroll
      for (int k = 0; k < U; ++k) u[i][k] = make_uint4(0, 0, 0, 0);
      if (on && in.x < 2 * rows) {
        const int row = in.x >> 1;
        const uint8_t *src = (in.x & 1 ? src_v + row * a.ldv : src_k + row * a.ldk) + in.head * kv.dim * 2;
        if (U == 1)
          u[i][0] = __ldg(reinterpret_cast<const uint4 *>(src));
        else
          load32(src, a.wide, u[i][0], u[i][U - 1]);
      }
      in.next(kv.heads);
    }
    if (turn == 0) {
      check_offsets(kv, s, a.T);
      locate_rows(kv, s, first, rows, tile, tok);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int row = to.x >> 1, which = to.x & 1, head = to.head;
      const long long at = row < rows ? tile[row] : -1;
      to.next(kv.heads);
      if (TYPE == LORA_KV_BF16) {
        if (at >= 0 && on) *held(kv.base + at, tok[row], which, head) = u[i][0];
        continue;
      }
      // the largest magnitude, as bits of bf16, two by two
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const uint4 v = u[i][k];
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
      }
      for (int d = a.lanes / 2; d; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(~0u, m, d));
      if (at < 0) continue;
      const Quant q = quant_of<TYPE == LORA_KV_E4M3 ? 448 : 127>(__uint_as_float(max(m >> 16, m & 0xffffu) << 16));
      uint32_t c[2 * U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float x[8];
        unpack8(u[i][k], x);
        c[2 * k] = code4<TYPE, true>(x, q);
        c[2 * k + 1] = code4<TYPE, true>(x + 4, q);
      }
      if (on) *held(kv.base + at, tok[row], which, head) = make_uint4(c[0], c[1], c[2 * U - 2], c[2 * U - 1]);
      if (part == 0) *held.scale(kv.base + at, tok[row], which, head) = q.scale;
    }
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks) kv_gather_kernel(KvView kv, KvSeqs s, RowArgs a) {
  constexpr int E = vec_elements(TYPE), kAhead = kGatherAhead;
  __shared__ long long tile[kMaxBlockRows];
  __shared__ int tok[kMaxBlockRows];
  const int first = blockIdx.x * a.rows, rows = min(a.rows, a.T - first);
  const int e = (threadIdx.x & (a.lanes - 1)) * E, step = kRowThreads / a.lanes;
  const HeldPlace<TYPE> held(kv, e);
  uint8_t *dst_k = a.k + first * a.ldk + e * 2, *dst_v = a.v + first * a.ldv + e * 2;
  RowWalk from(threadIdx.x / a.lanes, step, kv.heads), to = from;
  griddep_wait();
  griddep_launch_dependents();
  check_offsets(kv, s, a.T);
  locate_rows(kv, s, first, rows, tile, tok);
  __syncthreads();
  if (e >= kv.dim) return;
  while (from.x < 2 * rows) {
    uint4 u[kAhead];
    float scale[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int row = from.x >> 1, which = from.x & 1, head = from.head;
      const long long at = row < rows ? tile[row] : -1;
      from.next(kv.heads);
      u[i] = make_uint4(0, 0, 0, 0);
      scale[i] = 0.f;
      if (at < 0) continue;
      u[i] = *held(kv.base + at, tok[row], which, head);
      if (TYPE != LORA_KV_BF16) scale[i] = *held.scale(kv.base + at, tok[row], which, head);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int row = to.x >> 1, which = to.x & 1, head = to.head;
      to.next(kv.heads);
      if (row >= rows || tile[row] < 0) continue;
      uint8_t *dst = (which ? dst_v + row * a.ldv : dst_k + row * a.ldk) + head * kv.dim * 2;
      if (TYPE == LORA_KV_BF16) {
        __stcs(reinterpret_cast<uint4 *>(dst), u[i]);
        continue;
      }
      const uint32_t c[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      uint4 y[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[8];
        decode4<TYPE>(c[2 * k], x);
        decode4<TYPE>(c[2 * k + 1], x + 4);
        const float m = scale[i];
        y[k] = make_uint4(pack_bf16x2(x[0] * m, x[1] * m), pack_bf16x2(x[2] * m, x[3] * m),
                          pack_bf16x2(x[4] * m, x[5] * m), pack_bf16x2(x[6] * m, x[7] * m));
      }
      store32(dst, a.wide, y[0], y[1]);
    }
  }
}

// Reads and clears the status in one access: what another stream's call reports in
// between is in this reading or the next.
__global__ void kv_take_status_kernel(int *status, int *out) { *out = atomicExch(status, 0); }

}  // namespace lora

using namespace lora;

namespace {

bool shape_ok(int n_layers, int n_pages, int page_tokens, int heads, int dim, int type) {
  if (n_layers < 1 || n_layers > kKvMaxLayers || n_pages < 1) return false;
  if (page_tokens < kTileTokens || page_tokens > kKvMaxPageTokens || (page_tokens & (page_tokens - 1))) return false;
  if (heads < 1 || heads > kKvMaxHeads || dim < 16 || dim > kKvMaxDim || dim % 16) return false;
  return type == LORA_KV_BF16 || type == LORA_KV_E4M3 || type == LORA_KV_INT8;
}

long long page_bytes_of(int page_tokens, int heads, int dim, int type) {
  return (long long)heads * (page_tokens / kTileTokens) * kv_tile_bytes(type, dim);
}

// Checks of a row call (append, gather); LORA_OK with T == 0 means nothing to do.
int check_row_call(const lora_kv *kv, int layer, const void *k, int ldk, const void *v, int ldv,
                   const int32_t *table, int max_pages, const int32_t *lens, const int32_t *offsets, int n_seqs,
                   int T) {
  if (!kv || layer < 0 || layer >= kv->n_layers) return LORA_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxTokens || n_seqs < 0 || n_seqs > kMaxTokens || max_pages < 0) return LORA_ERR_INVALID_ARG;
  if (!offsets && n_seqs != T) return LORA_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0) return LORA_OK;
  if (!k || !v || !table || !lens || max_pages < 1) return LORA_ERR_INVALID_ARG;
  if (ldk < kv->heads * kv->dim || ldv < kv->heads * kv->dim) return LORA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || ldk % 8 || ldv % 8) return LORA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(offsets)) & 3)
    return LORA_ERR_ALIGNMENT;
  return LORA_OK;
}

// turns: at most so many rows to a block as its threads take in so many turns (0: no such limit).
template <class K>
int launch_rows(K kernel, const lora_kv *kv, int layer, const KvSeqs &s, RowArgs a, int turns, cudaStream_t st) {
  a.lanes = 1;
  while (a.lanes * vec_elements(kv->type) < kv->dim) a.lanes *= 2;
  a.wide = !((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) | a.ldk | a.ldv) & 31);
  const int at_once = kv->n_sm * kRowBlocks;
  a.rows = (a.T + at_once - 1) / at_once;
  if (turns) {
    const int vectors = turns * kGatherAhead * (kRowThreads / a.lanes), most = vectors / (2 * kv->heads);
    a.rows = a.rows > most ? (most > 0 ? most : 1) : a.rows;
  }
  a.rows = a.rows > kMaxBlockRows ? kMaxBlockRows : a.rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T + a.rows - 1) / a.rows);
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int rc = cuda_status(cudaLaunchKernelEx(&cfg, kernel, kv->view(layer), s, a));
  if (rc == LORA_OK) g_launches.fetch_add(1);
  return rc;
}

KvSeqs seqs_of(const int32_t *table, int max_pages, const int32_t *lens, const int32_t *offsets, int n) {
  KvSeqs s;
  s.table = table;
  s.lens = lens;
  s.offsets = offsets;
  s.max_pages = max_pages;
  s.n = n;
  return s;
}

int attend(lora_kv *kv, int layer, const void *q, int ldq, void *out, int ldo, float *lse, const float *sinks, int n_heads,
           const int32_t *page_table, int max_pages, const int32_t *seq_lens, int n_seqs, float scale, int window, void *ws,
           size_t ws_bytes, int stall, void *stream) {
  if (!kv || layer < 0 || layer >= kv->n_layers) return LORA_ERR_INVALID_ARG;
  if (n_heads < kv->heads || n_heads % kv->heads || n_heads > kKvMaxQHeads) return LORA_ERR_INVALID_ARG;
  if (n_seqs < 0 || n_seqs > kMaxTokens || max_pages < 0 || window < 0) return LORA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale > 0x1p100f) return LORA_ERR_INVALID_ARG;
  if (n_seqs == 0) return LORA_OK;
  if (!q || !out || !page_table || !seq_lens || !ws || max_pages < 1) return LORA_ERR_INVALID_ARG;
  const int width = n_heads * kv->dim;
  if (ldq < width || ldo < width) return LORA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(ws) || ldq % 8 || ldo % 8) return LORA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(sinks)) & 3)
    return LORA_ERR_ALIGNMENT;
  if (ws_bytes < attend_workspace_bytes(kv, n_heads)) return LORA_ERR_WORKSPACE;
  if (rows_overlap(q, size_t(ldq) * 2, size_t(width) * 2, n_seqs, out, size_t(ldo) * 2, size_t(width) * 2, n_seqs))
    return LORA_ERR_INVALID_ARG;
  AttendCall c;
  c.q = q;
  c.ldq = ldq;
  c.out = out;
  c.ldo = ldo;
  c.lse = lse;
  c.sinks = sinks;
  c.n_heads = n_heads;
  c.scale = scale;
  c.window = window;
  c.ws = ws;
  c.stall = stall;
  DeviceGuard g(kv->device);
  return launch_attend(kv, layer, seqs_of(page_table, max_pages, seq_lens, nullptr, n_seqs), c,
                       static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

size_t lora_kv_bytes_required(int n_layers, int n_pages, int page_tokens, int n_kv_heads, int head_dim, int kv_type) {
  if (!shape_ok(n_layers, n_pages, page_tokens, n_kv_heads, head_dim, kv_type)) return 0;
  const unsigned __int128 n = (unsigned __int128)page_bytes_of(page_tokens, n_kv_heads, head_dim, kv_type) * n_pages * n_layers;
  return n >> 62 ? 0 : (size_t)n;
}

int lora_kv_create(lora_kv **out, int device, int n_layers, int n_pages, int page_tokens, int n_kv_heads, int head_dim,
                   int kv_type, void *kv_mem, size_t kv_bytes) {
  if (!out) return LORA_ERR_INVALID_ARG;
  *out = nullptr;
  const size_t need = lora_kv_bytes_required(n_layers, n_pages, page_tokens, n_kv_heads, head_dim, kv_type);
  if (!need || !kv_mem || kv_bytes < need) return LORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(kv_mem) & 255u) return LORA_ERR_ALIGNMENT;
  int n_dev = 0;
  if (cuda_status(cudaGetDeviceCount(&n_dev)) != LORA_OK) return LORA_ERR_CUDA;
  if (device < 0 || device >= n_dev) return LORA_ERR_INVALID_ARG;
  lora_kv *kv = new (std::nothrow) lora_kv();
  if (!kv) return LORA_ERR_INVALID_ARG;
  kv->device = device;
  kv->n_layers = n_layers;
  kv->n_pages = n_pages;
  kv->page_tokens = page_tokens;
  while ((1 << kv->log2_page) < page_tokens) ++kv->log2_page;
  kv->heads = n_kv_heads;
  kv->dim = head_dim;
  kv->type = kv_type;
  kv->page_bytes = page_bytes_of(page_tokens, n_kv_heads, head_dim, kv_type);
  kv->layer_bytes = kv->page_bytes * n_pages;
  kv->mem = static_cast<uint8_t *>(kv_mem);
  DeviceGuard g(device);
  int rc = cuda_status(cudaDeviceGetAttribute(&kv->n_sm, cudaDevAttrMultiProcessorCount, device));
  if (rc == LORA_OK) rc = cuda_status(cudaMalloc(&kv->d_status, kKvStatusInts * sizeof(int)));
  if (rc == LORA_OK) {  // (on a stream that waits for no other: done before the first call on any)
    cudaStream_t st = nullptr;
    rc = cuda_status(cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking));
    if (rc == LORA_OK) rc = cuda_status(cudaMemsetAsync(kv->d_status, 0, kKvStatusInts * sizeof(int), st));
    if (rc == LORA_OK) rc = cuda_status(cudaStreamSynchronize(st));
    if (st) (void)cudaStreamDestroy(st);
  }
  if (rc == LORA_OK) rc = attend_setup(kv);
  if (rc != LORA_OK) {
    if (kv->d_status) (void)cudaFree(kv->d_status);
    delete kv;
    return rc;
  }
  *out = kv;
  return LORA_OK;
}

int lora_kv_destroy(lora_kv *kv) {
  if (!kv) return LORA_ERR_INVALID_ARG;
  int rc;
  {
    DeviceGuard g(kv->device);
    rc = cuda_status(cudaDeviceSynchronize());
    const int freed = cuda_status(cudaFree(kv->d_status));
    if (rc == LORA_OK) rc = freed;
  }
  delete kv;
  return rc;
}

int lora_kv_get_error(lora_kv *kv, int *device_status, void *stream) {
  if (!kv || !device_status) return LORA_ERR_INVALID_ARG;
  DeviceGuard g(kv->device);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int v = 0;
  int rc = cuda_status(cudaStreamSynchronize(st));  // (also refuses a stream that is being captured)
  if (rc == LORA_OK) {
    int *out = kv->d_status + 1 + kv->takes.fetch_add(1) % (kKvStatusInts - 1);
    kv_take_status_kernel<<<1, 1, 0, st>>>(kv->d_status, out);
    rc = cuda_status(cudaGetLastError());
    if (rc == LORA_OK) g_launches.fetch_add(1);
    if (rc == LORA_OK) rc = cuda_status(cudaMemcpyAsync(&v, out, 4, cudaMemcpyDeviceToHost, st));
    if (rc == LORA_OK) rc = cuda_status(cudaStreamSynchronize(st));
  }
  if (rc == LORA_OK) *device_status = v;
  return rc;
}

int lora_kv_append(lora_kv *kv, int layer, const void *k, int ldk, const void *v, int ldv, const int32_t *page_table,
                   int max_pages, const int32_t *seq_lens, const int32_t *row_offsets, int n_seqs, int T,
                   void *stream) {
  NvtxRange nvtx_range("lora_kv_append");
  int rc = check_row_call(kv, layer, k, ldk, v, ldv, page_table, max_pages, seq_lens, row_offsets, n_seqs, T);
  if (rc != LORA_OK || T == 0 || n_seqs == 0) return rc;
  RowArgs a = {};
  a.k = static_cast<uint8_t *>(const_cast<void *>(k));
  a.v = static_cast<uint8_t *>(const_cast<void *>(v));
  a.ldk = 2ll * ldk;
  a.ldv = 2ll * ldv;
  a.T = T;
  DeviceGuard g(kv->device);
  const KvSeqs s = seqs_of(page_table, max_pages, seq_lens, row_offsets, n_seqs);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (kv->type == LORA_KV_BF16) return launch_rows(kv_append_kernel<LORA_KV_BF16>, kv, layer, s, a, 0, st);
  if (kv->type == LORA_KV_E4M3) return launch_rows(kv_append_kernel<LORA_KV_E4M3>, kv, layer, s, a, 0, st);
  return launch_rows(kv_append_kernel<LORA_KV_INT8>, kv, layer, s, a, 0, st);
}

int lora_kv_gather(lora_kv *kv, int layer, void *k, int ldk, void *v, int ldv, const int32_t *page_table,
                   int max_pages, const int32_t *seq_lens, const int32_t *row_offsets, int n_seqs, int T,
                   void *stream) {
  NvtxRange nvtx_range("lora_kv_gather");
  int rc = check_row_call(kv, layer, k, ldk, v, ldv, page_table, max_pages, seq_lens, row_offsets, n_seqs, T);
  if (rc != LORA_OK || T == 0 || n_seqs == 0) return rc;
  const size_t width = size_t(kv->heads) * kv->dim * 2;
  if (rows_overlap(k, size_t(ldk) * 2, width, T, v, size_t(ldv) * 2, width, T)) return LORA_ERR_INVALID_ARG;
  RowArgs a = {};
  a.k = static_cast<uint8_t *>(k);
  a.v = static_cast<uint8_t *>(v);
  a.ldk = 2ll * ldk;
  a.ldv = 2ll * ldv;
  a.T = T;
  DeviceGuard g(kv->device);
  const KvSeqs s = seqs_of(page_table, max_pages, seq_lens, row_offsets, n_seqs);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (kv->type == LORA_KV_BF16) return launch_rows(kv_gather_kernel<LORA_KV_BF16>, kv, layer, s, a, kGatherTurns, st);
  if (kv->type == LORA_KV_E4M3) return launch_rows(kv_gather_kernel<LORA_KV_E4M3>, kv, layer, s, a, kGatherTurns, st);
  return launch_rows(kv_gather_kernel<LORA_KV_INT8>, kv, layer, s, a, kGatherTurns, st);
}

size_t lora_attend_workspace_bytes(const lora_kv *kv, int n_heads) {
  if (!kv || n_heads < kv->heads || n_heads % kv->heads || n_heads > kKvMaxQHeads) return 0;
  return attend_workspace_bytes(kv, n_heads);
}

int lora_attend(lora_kv *kv, int layer, const void *q, int ldq, void *out, int ldo, float *lse, const float *sinks,
                int n_heads, const int32_t *page_table, int max_pages, const int32_t *seq_lens, int n_seqs, float scale,
                int window, void *ws, size_t ws_bytes, void *stream) {
  NvtxRange nvtx_range("lora_attend");
  return attend(kv, layer, q, ldq, out, ldo, lse, sinks, n_heads, page_table, max_pages, seq_lens, n_seqs, scale, window,
                ws, ws_bytes, 0, stream);
}

int lora_selftest_stalled_attend(lora_kv *kv, int layer, const void *q, int ldq, void *out, int ldo, int n_heads,
                                 const int32_t *page_table, int max_pages, const int32_t *seq_lens, int n_seqs, void *ws,
                                 size_t ws_bytes, void *stream) {
  NvtxRange nvtx_range("lora_selftest_stalled_attend");
  return attend(kv, layer, q, ldq, out, ldo, nullptr, nullptr, n_heads, page_table, max_pages, seq_lens, n_seqs, 1.f, 0,
                ws, ws_bytes, kStallAll, stream);
}

int lora_selftest_late_lane_attend(lora_kv *kv, int layer, const void *q, int ldq, void *out, int ldo, int n_heads,
                                   const int32_t *page_table, int max_pages, const int32_t *seq_lens, int n_seqs, void *ws,
                                   size_t ws_bytes, int lane, void *stream) {
  NvtxRange nvtx_range("lora_selftest_late_lane_attend");
  if (lane < 0 || lane > 31) return LORA_ERR_INVALID_ARG;
  return attend(kv, layer, q, ldq, out, ldo, nullptr, nullptr, n_heads, page_table, max_pages, seq_lens, n_seqs, 1.f, 0,
                ws, ws_bytes, kStallLane + lane, stream);
}

}  // extern "C"
