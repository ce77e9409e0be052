// kv.cu -- the paged key/value cache: handle, quantising append, read-back.
//
// The cache lives in pages of caller-owned memory located through a page table,
// the unified paging of "Multi-LoRA Serving: Sharing One GPU Across Adapters"
// (section "How S-LoRA Proved the Model") for the other half of what a serving
// GPU holds.  append writes new keys and values (held as bf16, e4m3 or int8,
// kv.cuh), gather reads held rows back as bf16.  Both are one pass over their
// bytes; what bounds them is HBM.
//
// Work split: a row of one head's K or V is handled by `lanes` neighbouring
// threads (a power of two, 8 elements or 16 bytes of bf16 each), which reduce
// its largest magnitude with shuffles and store 8 or 16 bytes each into the
// token's tile.  A block takes `rows` consecutive rows of the batch (about four
// vectors per thread); its warps first look up each row's sequence (a 32-way
// search in row_offsets: two dependent reads up to 1024 sequences) and page.
#include <new>

#include "kv.cuh"

namespace lora {

constexpr int kRowThreads = 256;
constexpr int kMaxBlockRows = 64;

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
  for (int i = warp; i < rows; i += kRowThreads / 32) {
    const int t = first + i;
    int seq = t, back = 1, own = 1;  // the row's distance from its sequence's end; the sequence's rows
    if (s.offsets) {
      seq = find_seq(s.offsets, s.n, t);
      if (seq >= 0) {
        const int end = __ldg(s.offsets + seq + 1);
        back = end - t;
        own = end - __ldg(s.offsets + seq);
      }
    }
    if (lane) continue;
    long long at = -1;
    int row = 0;
    if (seq >= 0) {
      const int len = s.lens[seq];
      const bool none = len == -1 || (len == 0 && !s.offsets);
      if (!none) {
        if (len > 0 && len <= ((long long)s.max_pages << kv.log2_page) && own <= len) {
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
  int lanes;          // threads per vector (power of two >= dim / 8)
};

// Vector w of a block: (row, K or V, head), heads fastest, as the rows lie in memory.
struct RowVec {
  int row, which, head;
};
__device__ __forceinline__ RowVec row_vec(int w, int heads) {
  RowVec r;
  r.head = w % heads;
  const int x = w / heads;
  r.which = x & 1;
  r.row = x >> 1;
  return r;
}

template <int TYPE>
__device__ __forceinline__ uint8_t *held_at(const KvView &kv, long long tile, int tok, const RowVec &r, int e) {
  constexpr int ES = kv_elt(TYPE);
  const int row_bytes = kv.dim * ES, b = e * ES;
  uint8_t *t = kv.base + tile + r.head * kv_head_stride(kv) + (r.which * kTileTokens + tok) * row_bytes;
  return t + kv_chunk(b / 16, tok, row_bytes / 16) * 16 + b % 16;
}
__device__ __forceinline__ float *scale_at(const KvView &kv, long long tile, int tok, const RowVec &r) {
  uint8_t *t = kv.base + tile + r.head * kv_head_stride(kv) + 2 * kTileTokens * kv.dim;
  return reinterpret_cast<float *>(t) + r.which * kTileTokens + tok;
}

template <int TYPE>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(KvView kv, KvSeqs s, RowArgs a) {
  __shared__ long long tile[kMaxBlockRows];
  __shared__ int tok[kMaxBlockRows];
  griddep_wait();
  griddep_launch_dependents();
  const int first = blockIdx.x * a.rows, rows = min(a.rows, a.T - first);
  check_offsets(kv, s, a.T);
  locate_rows(kv, s, first, rows, tile, tok);
  __syncthreads();
  const int part = threadIdx.x & (a.lanes - 1), e = part * 8;
  const int n = rows * 2 * kv.heads;
  // (whole groups of lanes leave the loop together, but a warp may not: the
  // shuffles name the group's own lanes only)
  const unsigned group = (a.lanes == 32 ? ~0u : ((1u << a.lanes) - 1u) << (threadIdx.x & 31 & ~(a.lanes - 1)));
  for (int w = threadIdx.x / a.lanes; w < n; w += kRowThreads / a.lanes) {
    const RowVec r = row_vec(w, kv.heads);
    if (tile[r.row] < 0) continue;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (e < kv.dim) {
      const uint8_t *src = r.which ? a.v + (first + r.row) * a.ldv : a.k + (first + r.row) * a.ldk;
      u = __ldg(reinterpret_cast<const uint4 *>(src + (r.head * kv.dim + e) * 2));
    }
    if (TYPE == LORA_KV_BF16) {
      if (e < kv.dim) *reinterpret_cast<uint4 *>(held_at<TYPE>(kv, tile[r.row], tok[r.row], r, e)) = u;
    } else {
      float x[8];
      unpack8(u, x);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
      for (int d = a.lanes / 2; d; d >>= 1) m = max(m, __shfl_xor_sync(group, m, d));
      const Quant q = quant_of<TYPE == LORA_KV_E4M3 ? 448 : 127>(__uint_as_float(m));
      if (e < kv.dim)
        *reinterpret_cast<uint2 *>(held_at<TYPE>(kv, tile[r.row], tok[r.row], r, e)) =
            make_uint2(code4<TYPE>(x, q), code4<TYPE>(x + 4, q));
      if (part == 0) *scale_at(kv, tile[r.row], tok[r.row], r) = q.scale;
    }
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kRowThreads) kv_gather_kernel(KvView kv, KvSeqs s, RowArgs a) {
  __shared__ long long tile[kMaxBlockRows];
  __shared__ int tok[kMaxBlockRows];
  griddep_wait();
  griddep_launch_dependents();
  const int first = blockIdx.x * a.rows, rows = min(a.rows, a.T - first);
  check_offsets(kv, s, a.T);
  locate_rows(kv, s, first, rows, tile, tok);
  __syncthreads();
  const int e = (threadIdx.x & (a.lanes - 1)) * 8;
  const int n = rows * 2 * kv.heads;
  if (e >= kv.dim) return;
  for (int w = threadIdx.x / a.lanes; w < n; w += kRowThreads / a.lanes) {
    const RowVec r = row_vec(w, kv.heads);
    if (tile[r.row] < 0) continue;
    const uint8_t *src = held_at<TYPE>(kv, tile[r.row], tok[r.row], r, e);
    uint4 u;
    if (TYPE == LORA_KV_BF16) {
      u = *reinterpret_cast<const uint4 *>(src);
    } else {
      const uint2 c = *reinterpret_cast<const uint2 *>(src);
      const float scale = *scale_at(kv, tile[r.row], tok[r.row], r);
      float x[8];
      decode4<TYPE>(c.x, x);
      decode4<TYPE>(c.y, x + 4);
      u.x = pack_bf16x2(x[0] * scale, x[1] * scale);
      u.y = pack_bf16x2(x[2] * scale, x[3] * scale);
      u.z = pack_bf16x2(x[4] * scale, x[5] * scale);
      u.w = pack_bf16x2(x[6] * scale, x[7] * scale);
    }
    uint8_t *dst = r.which ? a.v + (first + r.row) * a.ldv : a.k + (first + r.row) * a.ldk;
    *reinterpret_cast<uint4 *>(dst + (r.head * kv.dim + e) * 2) = u;
  }
}

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

template <class K>
int launch_rows(K kernel, const lora_kv *kv, int layer, const KvSeqs &s, RowArgs a, cudaStream_t st) {
  a.lanes = 2;
  while (a.lanes * 8 < kv->dim) a.lanes *= 2;
  const int per_row = 2 * kv->heads * a.lanes;
  a.rows = 4 * kRowThreads / per_row;
  a.rows = a.rows < 1 ? 1 : a.rows > kMaxBlockRows ? kMaxBlockRows : a.rows;
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
  if (rc == LORA_OK) rc = cuda_status(cudaMalloc(&kv->d_status, 256));
  if (rc == LORA_OK) rc = cuda_status(cudaMemset(kv->d_status, 0, 256));
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
  int v = 0;
  int rc = cuda_status(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  if (rc == LORA_OK) rc = cuda_status(cudaMemcpy(&v, kv->d_status, 4, cudaMemcpyDeviceToHost));
  if (rc == LORA_OK) rc = cuda_status(cudaMemset(kv->d_status, 0, 4));
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
  if (kv->type == LORA_KV_BF16) return launch_rows(kv_append_kernel<LORA_KV_BF16>, kv, layer, s, a, st);
  if (kv->type == LORA_KV_E4M3) return launch_rows(kv_append_kernel<LORA_KV_E4M3>, kv, layer, s, a, st);
  return launch_rows(kv_append_kernel<LORA_KV_INT8>, kv, layer, s, a, st);
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
  if (kv->type == LORA_KV_BF16) return launch_rows(kv_gather_kernel<LORA_KV_BF16>, kv, layer, s, a, st);
  if (kv->type == LORA_KV_E4M3) return launch_rows(kv_gather_kernel<LORA_KV_E4M3>, kv, layer, s, a, st);
  return launch_rows(kv_gather_kernel<LORA_KV_INT8>, kv, layer, s, a, st);
}

size_t lora_attend_workspace_bytes(const lora_kv *kv, int n_heads) {
  if (!kv || n_heads < kv->heads || n_heads % kv->heads) return 0;
  return attend_workspace_bytes(kv, n_heads);
}

int lora_attend(lora_kv *kv, int layer, const void *q, int ldq, void *out, int ldo, float *lse, const float *sinks,
                int n_heads, const int32_t *page_table, int max_pages, const int32_t *seq_lens, int n_seqs, float scale,
                int window, void *ws, size_t ws_bytes, void *stream) {
  NvtxRange nvtx_range("lora_attend");
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
  DeviceGuard g(kv->device);
  return launch_attend(kv, layer, seqs_of(page_table, max_pages, seq_lens, nullptr, n_seqs), c,
                       static_cast<cudaStream_t>(stream));
}

}  // extern "C"
