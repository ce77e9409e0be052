// kv.cuh -- the paged key/value cache: layout, device view, quantisation.
//
// Per layer the cache is a stack of pages of page_tokens tokens.  A page holds,
// head after head, tiles of 16 tokens; one tile is everything a 16-token step
// of the attention needs of one head, in one contiguous range:
//     [K: 16 rows of dim][V: 16 rows of dim]            bf16 caches
//     [K][V][16 fp32 K scales][16 fp32 V scales]        8-bit caches
// so that the attention fetches it with a single bulk copy.  Inside a row the
// 16-byte chunks are permuted (kv_chunk): the eight rows of an ldmatrix then
// fall into different shared-memory banks with no padding and no staging pass.
#pragma once

#include <atomic>

#include "internal.cuh"

namespace lora {

constexpr int kTileTokens = 16;
constexpr int kKvMaxDim = 256;
constexpr int kKvMaxHeads = 1024;   // key heads
constexpr int kKvMaxQHeads = 4096;  // query heads
constexpr int kKvMaxLayers = 4096;
constexpr int kKvMaxPageTokens = 1024;
constexpr int kKvStatusInts = 64;

__host__ __device__ constexpr int kv_elt(int type) { return type == LORA_KV_BF16 ? 2 : 1; }
__host__ __device__ constexpr int kv_row_bytes(int type, int dim) { return dim * kv_elt(type); }
__host__ __device__ constexpr int kv_tile_bytes(int type, int dim) {
  return 2 * kTileTokens * kv_row_bytes(type, dim) + (type == LORA_KV_BF16 ? 0 : 2 * kTileTokens * 4);
}

// Position of 16-byte chunk c in row r of `chunks` chunks.  With g the largest
// power of two (at most 8) that divides `chunks`, eight consecutive rows start
// at 8 / g different bank groups, each shared by g rows; xor-ing the row's
// number within its group into the chunk's low bits separates those g.
__host__ __device__ constexpr int kv_chunk(int c, int r, int chunks) {
  const int low = chunks & -chunks, g = low < 8 ? low : 8;
  return c ^ ((r / (8 / g)) & (g - 1));
}

// Device view of one layer of a cache.
struct KvView {
  uint8_t *base;         // the layer's first page
  long long page_bytes;  // of one page (all heads)
  int tile_bytes;
  int n_pages;
  int log2_page;         // tokens per page
  int heads, dim;
  int *status;
};

// One call's sequences: their pages, their lengths and, for row calls, which
// rows are whose (row_offsets null: row s belongs to sequence s).
struct KvSeqs {
  const int32_t *table;
  const int32_t *lens;
  const int32_t *offsets;
  int max_pages;
  int n;
};

// A length that the table has room for, and that leaves positions room in 32 bits.
constexpr int kKvMaxLen = 1 << 30;
__device__ __forceinline__ bool kv_len_ok(const KvView &kv, const KvSeqs &s, int len) {
  return len <= kKvMaxLen && len <= ((long long)s.max_pages << kv.log2_page);
}

// Byte offset of a token's tile of head 0 from the layer's base, -1 where the
// page number is not one of the cache's.
__device__ __forceinline__ long long kv_tile_offset(const KvView &kv, int page, int pos) {
  if (page < 0 || page >= kv.n_pages) return -1;
  const int sub = (pos & ((1 << kv.log2_page) - 1)) / kTileTokens;
  return page * kv.page_bytes + (long long)sub * kv.tile_bytes;
}
__device__ __forceinline__ long long kv_head_stride(const KvView &kv) {
  return (long long)kv.tile_bytes << (kv.log2_page - 4);
}

// ------------------------------------------------------------ quantisation
//
// A row of values (a token's key or value of one head; a norm's row or group)
// is held as codes and one fp32 scale:
//     scale = amax / qmax,   code = round_to_nearest_even(x * qmax / amax),
// qmax = 448 (e4m3) or 127 (int8).  The quotient of two bf16 values often lies
// exactly half way between two codes, so such a quotient has to come out exact:
// the product with qmax is exact for bf16 x, the residual of a first quotient is
// exact by fma, and the quotient corrected with it rounds to the exact one where
// that is representable (an approximate reciprocal of amax suffices for both).
// Every other quotient of bf16 values is further from a tie than fp32's error.
// The scale's division by a constant is corrected in the same way.  From amax
// 2^64 on both sides are scaled by 2^-64, which keeps the product and the
// reciprocal in range.  A row whose largest magnitude is below 2^-100 is held as
// zeros with scale 0 (its scale would lose its bits to underflow); one with an
// infinity or a NaN has a NaN for its scale, so that all its values read back as
// NaN.
struct Quant {
  float scale;  // what the codes are multiplied by when read
  float mul;    // qmax, times 2^-64 from amax 2^64 on
  float amax;   // in the same scaling
  float rcp;    // about 1 / amax
};

template <int QMAX>
__device__ __forceinline__ Quant quant_of(float amax) {
  Quant q;
  const bool none = amax < 0x1p-100f, big = amax >= 0x1p64f;
  constexpr float kInv = 1.f / QMAX;
  const float s = amax * kInv;
  q.scale = none ? 0.f : fmaf(fmaf(-s, (float)QMAX, amax), kInv, s);  // (an infinity: inf - inf)
  q.amax = big ? amax * 0x1p-64f : amax;
  q.mul = none ? 0.f : big ? QMAX * 0x1p-64f : (float)QMAX;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.rcp) : "f"(q.amax));
  if (none) q.rcp = 0.f;
  return q;
}
// x * qmax / amax, and the same for two values with the packed fp32 instructions,
// half as many (append of 4096 rows, 32 heads of 128: 25.1 and 27.3 us; the
// norm has no registers left for the pairs: 48.7 and 50.1 us for 8192 x 4096).
__device__ __forceinline__ float quant_div(float x, const Quant &q) {
  const float a = x * q.mul, t = a * q.rcp;
  return fmaf(fmaf(-t, q.amax, a), q.rcp, t);
}
__device__ __forceinline__ unsigned long long pair2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float2 quant_div(float x, float y, const Quant &q) {
  const unsigned long long rcp = pair2(q.rcp, q.rcp);
  const unsigned long long a = mul2(pair2(x, y), pair2(q.mul, q.mul)), t = mul2(a, rcp);
  const unsigned long long z = fma2(fma2(t, pair2(-q.amax, -q.amax), a), rcp, t);
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(z));
  return r;
}

// Two fp32 values as two e4m3 bytes (nearest even, values past 448 as 448, NaN kept).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four fp32 values as four int8 bytes (nearest even, at most +-127, NaN as 0).
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
  const int i = min(127, max(-127, __float2int_rn(a))), j = min(127, max(-127, __float2int_rn(b)));
  const int k = min(127, max(-127, __float2int_rn(c))), l = min(127, max(-127, __float2int_rn(d)));
  return (i & 255) | (j & 255) << 8 | (k & 255) << 16 | (uint32_t)(l & 255) << 24;
}
template <int TYPE, bool PAIRS>
__device__ __forceinline__ uint32_t code4(const float *x, const Quant &q) {
  float2 lo, hi;
  if (PAIRS) {
    lo = quant_div(x[0], x[1], q);
    hi = quant_div(x[2], x[3], q);
  } else {
    lo = make_float2(quant_div(x[0], q), quant_div(x[1], q));
    hi = make_float2(quant_div(x[2], q), quant_div(x[3], q));
  }
  if (TYPE == LORA_KV_E4M3) return e4m3x2(lo.x, lo.y) | e4m3x2(hi.x, hi.y) << 16;
  return int8x4(lo.x, lo.y, hi.x, hi.y);
}

// Four held bytes as the numbers they encode (before the scale).
template <int TYPE>
__device__ __forceinline__ void decode4(uint32_t w, float *x) {
  if (TYPE == LORA_KV_E4M3) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t f;  // two fp16
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)(w >> (16 * h))));
      asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
          : "=f"(x[2 * h]), "=f"(x[2 * h + 1])
          : "r"(f));
    }
  } else {
#pragma unroll
    for (int b = 0; b < 4; ++b) x[b] = (float)(int8_t)(w >> (8 * b));
  }
}

}  // namespace lora

// ---------------------------------------------------------------- host cache
struct lora_kv {
  int device = 0;
  int n_layers = 0, n_pages = 0, page_tokens = 0, log2_page = 0, heads = 0, dim = 0, type = 0;
  long long page_bytes = 0, layer_bytes = 0;
  uint8_t *mem = nullptr;
  int *d_status = nullptr;  // [kKvStatusInts]: the status, then places for readings of it
  std::atomic<unsigned> takes{0};
  int n_sm = 0;

  lora::KvView view(int layer) const {
    lora::KvView v;
    v.base = mem + layer * layer_bytes;
    v.page_bytes = page_bytes;
    v.tile_bytes = lora::kv_tile_bytes(type, dim);
    v.n_pages = n_pages;
    v.log2_page = log2_page;
    v.heads = heads;
    v.dim = dim;
    v.status = d_status;
    return v;
  }
};

namespace lora {

// Whether rows a [rows_a, width_a of lda bytes] and b share a byte.  Rows of
// the same pitch may interleave (column slices of one buffer).
inline bool rows_overlap(const void *a, size_t lda, size_t width_a, int rows_a, const void *b, size_t ldb,
                         size_t width_b, int rows_b) {
  if (!a || !b || rows_a < 1 || rows_b < 1) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const uintptr_t xe = x + size_t(rows_a - 1) * lda + width_a, ye = y + size_t(rows_b - 1) * ldb + width_b;
  if (xe <= y || ye <= x) return false;
  if (lda != ldb || !lda) return true;
  const size_t m = y >= x ? (y - x) % lda : (lda - (x - y) % lda) % lda;  // b's column in a's rows
  return m < width_a || m + width_b > lda;
}

inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return LORA_OK;
  (void)cudaGetLastError();
  return LORA_ERR_CUDA;
}

int attend_setup(lora_kv *kv);
// What the self-tests stall: nothing is fetched, so that every wait runs out; or one
// lane of each warp finds its waits run out from the warp's third step on.
enum { kStallAll = 1, kStallLane = 2 };

struct AttendCall {
  const void *q;
  int ldq;
  void *out;
  int ldo;
  float *lse;
  const float *sinks;
  int n_heads;
  float scale;
  int window;
  void *ws;
  int stall;  // test only: 0, kStallAll, or kStallLane + a lane
};
int launch_attend(const lora_kv *kv, int layer, const KvSeqs &s, const AttendCall &c, cudaStream_t st);
size_t attend_workspace_bytes(const lora_kv *kv, int n_heads);

}  // namespace lora
