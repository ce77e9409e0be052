// norm.cu -- the residual's addition and the root-mean-square norm before an
// adapted projection, in one pass:
//     h = x + residual,  n = h / sqrt(mean(h^2) + eps) * weight,
// written as bf16(h) (the next residual), bf16(n) (the rows that lora_linear
// and lora_apply read) and e4m3 codes of n with one fp32 scale per row or per
// group of columns (the rows of a base product in 8 bits; quantisation as the
// key/value cache's, kv.cuh).  h and n stay in fp32 between the roundings: a
// row is read once into registers, and every output is rounded once from them.
//
// Bound by HBM: 9 bytes per element in the full form.  A row is held by `tpr`
// threads, VPT 16-byte vectors each, vector lane + i * tpr to keep the loads
// contiguous; rows of at most 32 vectors share a warp, longer ones take whole
// warps that meet in shared memory once for the sum of squares and, with a
// scale per row, once for the largest magnitude.  A group's lanes are
// neighbours in a warp, so its scale needs no shared memory.  Four vectors a
// thread where there are many rows: few threads then wait at a row's two meetings
// and an SM has 100 KB on their way (8192 x 4096 in the full form, passes of a graph:
// 48.7 us, 95 % of a copy's rate, though a thread spills 24 bytes; two vectors
// 54.7 us, one 70.4); two where rows are fewer than four to an SM and the time is
// one row's latency (one row 2.3 us, 512 4.3; four vectors 2.7 and 4.7).  Rows of 33
// to 128 vectors are blocks of one warp, 32 to an SM at most (16384 x 512 with y alone:
// 18 us for 34 MB).
#include "kv.cuh"

namespace lora {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxVpt = 4;
constexpr int kNormMaxWidth = 8 * kNormMaxThreads * kNormMaxVpt;

struct NormArgs {
  const uint8_t *x, *res, *weight;
  uint8_t *sum, *y, *q;
  float *scales;
  long long ldx, ldr, lds, ldy, ldq;  // bytes
  float eps;
  int group, log2_vecs;  // columns of a scale (0: the row), and log2 of its vectors
  int T, d;
  int tpr;    // threads per row
};

// The larger of two, a NaN where either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int VPT>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(NormArgs a) {
  __shared__ float part[32];
  __shared__ uint32_t peak[32];
  const int slot = threadIdx.x / a.tpr, lane = threadIdx.x - slot * a.tpr;
  const long long row = (long long)blockIdx.x * (blockDim.x / a.tpr) + slot;
  const int nv = a.d / 8, nw = a.tpr / 32;  // nw: warps of a row (0 when rows share one)
  const bool live = row < a.T;
  // a thread's place in each operand; its vectors are `hop` bytes apart (half that in q)
  const int hop = a.tpr * 16;
  const uint8_t *x = a.x + row * a.ldx + lane * 16, *res = a.res ? a.res + row * a.ldr + lane * 16 : nullptr;
  const uint8_t *weight = a.weight + lane * 16;
  uint8_t *sum = a.sum ? a.sum + row * a.lds + lane * 16 : nullptr, *y = a.y ? a.y + row * a.ldy + lane * 16 : nullptr;
  uint8_t *qs = a.q + row * a.ldq + lane * 8;
  griddep_wait();
  griddep_launch_dependents();
  float h[VPT][8];
  uint4 xs[VPT], rs[VPT], w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = lane + i * a.tpr;
    xs[i] = rs[i] = w[i] = make_uint4(0, 0, 0, 0);
    if (live && v < nv) {
      w[i] = __ldg(reinterpret_cast<const uint4 *>(weight + i * hop));
      xs[i] = *reinterpret_cast<const uint4 *>(x + i * hop);
      if (res) rs[i] = *reinterpret_cast<const uint4 *>(res + i * hop);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float r[8];
    unpack8(xs[i], h[i]);
    unpack8(rs[i], r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] += r[e];
      ss = fmaf(h[i][e], h[i][e], ss);
    }
  }
  const int width = min(a.tpr, 32);
  auto row_sum = [&](float x) {
    for (int d = width / 2; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    if (nw > 1) {
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
      __syncthreads();
      x = 0.f;
      for (int i = 0; i < nw; ++i) x += part[slot * nw + i];
    }
    return x;
  };
  ss = row_sum(ss);
  const float mean = ss / a.d + a.eps;
  float inv = __fdiv_rn(1.f, __fsqrt_rn(mean));
  // Squares past fp32's range (h from 2^56 on), or too small for its bits with no eps
  // above them: once more in units that bring them back (all warps of a row agree).
  // Small h are brought to their unit before the product too, since 1 / rms may pass
  // the range; large ones are not, since a row's smallest would lose bits.
  bool small = false;
  const bool far = !(mean >= 0x1p-100f && mean < INFINITY);
  if (__builtin_expect(__any_sync(~0u, far), 0)) {
    small = mean < 0x1p-100f;
    const float unit = small ? 0x1p80f : far ? 0x1p-80f : 1.f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = h[i][e] * unit;
        ss = fmaf(t, t, ss);
      }
    if (nw > 1) __syncthreads();  // (part has been read)
    ss = row_sum(ss);
    inv = __fdiv_rn(1.f, __fsqrt_rn(ss / a.d + a.eps * unit * unit)) * fminf(unit, 1.f);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = lane + i * a.tpr;
    if (live && v < nv && sum)
      *reinterpret_cast<uint4 *>(sum + i * hop) =
          make_uint4(pack_bf16x2(h[i][0], h[i][1]), pack_bf16x2(h[i][2], h[i][3]), pack_bf16x2(h[i][4], h[i][5]),
                     pack_bf16x2(h[i][6], h[i][7]));
    if (__builtin_expect(small, 0)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] *= 0x1p80f;
    }
    float g[8];
    unpack8(w[i], g);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * inv * g[e];
    if (live && v < nv && y)
      *reinterpret_cast<uint4 *>(y + i * hop) =
          make_uint4(pack_bf16x2(h[i][0], h[i][1]), pack_bf16x2(h[i][2], h[i][3]), pack_bf16x2(h[i][4], h[i][5]),
                     pack_bf16x2(h[i][6], h[i][7]));
  }
  if (!a.q) return;  // (the same for the whole grid)
  float *scales = a.scales + row * (a.group ? nv >> a.log2_vecs : 1);
  uint32_t m[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    // (past the row x, residual and weight are 0, and so is h, unless the row's inv is not finite)
    float top = fabsf(h[i][0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) top = max_nan(top, fabsf(h[i][e]));
    m[i] = lane + i * a.tpr < nv ? __float_as_uint(top) & 0x7fffffffu : 0u;
  }
  if (a.group) {
    const int lanes = a.group / 8;
    if (lanes >= 16) {  // one or two reductions of the warp's hardware
      const unsigned who = lanes == 32 ? ~0u : 0xffffu << (threadIdx.x & 16);
#pragma unroll
      for (int i = 0; i < VPT; ++i) m[i] = __reduce_max_sync(who, m[i]);
    } else {
      for (int d = lanes / 2; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < VPT; ++i) m[i] = max(m[i], __shfl_xor_sync(~0u, m[i], d));
    }
  } else {
#pragma unroll
    for (int i = 1; i < VPT; ++i) m[0] = max(m[0], m[i]);
    for (int d = width / 2; d; d >>= 1) m[0] = max(m[0], __shfl_xor_sync(~0u, m[0], d));
    if (nw > 1) {
      if ((threadIdx.x & 31) == 0) peak[threadIdx.x >> 5] = m[0];
      __syncthreads();
      m[0] = 0;
      for (int i = 0; i < nw; ++i) m[0] = max(m[0], peak[slot * nw + i]);
    }
#pragma unroll
    for (int i = 1; i < VPT; ++i) m[i] = m[0];
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = lane + i * a.tpr;
    if (!live || v >= nv) continue;
    const Quant q = quant_of<448>(__uint_as_float(m[i]));
    *reinterpret_cast<uint2 *>(qs + i * (hop / 2)) =
        make_uint2(code4<LORA_KV_E4M3, false>(h[i], q), code4<LORA_KV_E4M3, false>(h[i] + 4, q));
    if (a.group) {
      if ((v & ((1 << a.log2_vecs) - 1)) == 0) scales[v >> a.log2_vecs] = q.scale;
    } else if (v == 0) {
      *scales = q.scale;
    }
  }
}

template <int VPT>
static int launch_norm(const NormArgs &a, int rows_per_block, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + rows_per_block - 1) / rows_per_block));
  cfg.blockDim = dim3(a.tpr * rows_per_block);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int rc = cuda_status(cudaLaunchKernelEx(&cfg, rmsnorm_kernel<VPT>, a));
  if (rc == LORA_OK) g_launches.fetch_add(1);
  return rc;
}

// Operands that are written must not share bytes with one another or with the
// weight; an output may be an input's own rows (same address and pitch: a row
// is in registers before any of it is written) but not overlap it otherwise.
struct NormRows {
  const void *p;
  size_t ld, width;
};
static bool clash(const NormRows &out, const NormRows &in, int T) {
  if (out.p && out.p == in.p && out.ld == in.ld) return false;
  return rows_overlap(out.p, out.ld, out.width, T, in.p, in.ld, in.width, T);
}

}  // namespace lora

using namespace lora;

extern "C" {

int lora_rmsnorm(int device, const void *x, int ldx, const void *residual, int ldr, void *residual_out, int ldro,
                 const void *weight, float eps, void *y, int ldy, void *q, int ldq, float *q_scales, int group, int T,
                 int d, void *stream) {
  NvtxRange nvtx_range("lora_rmsnorm");
  if (T < 0 || T > kMaxTokens || d < 8 || d > kNormMaxWidth || !(eps >= 0.f)) return LORA_ERR_INVALID_ARG;
  if (d % 8) return LORA_ERR_ALIGNMENT;
  if (group < 0 || (group && (group < 16 || group > 256 || (group & (group - 1)) || d % group)))
    return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!x || !weight || (!y && !q) || (q && !q_scales)) return LORA_ERR_INVALID_ARG;
  if (ldx < d || (residual && ldr < d) || (residual_out && ldro < d) || (y && ldy < d) || (q && ldq < d))
    return LORA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(weight) || !aligned16(residual) || !aligned16(residual_out) || !aligned16(y) ||
      !aligned16(q) || (reinterpret_cast<uintptr_t>(q_scales) & 3))
    return LORA_ERR_ALIGNMENT;
  if (ldx % 8 || (residual && ldr % 8) || (residual_out && ldro % 8) || (y && ldy % 8) || (q && ldq % 8))
    return LORA_ERR_ALIGNMENT;
  const size_t w2 = size_t(d) * 2;
  const NormRows in[2] = {{x, size_t(ldx) * 2, w2}, {residual, size_t(ldr) * 2, w2}};
  const size_t n_scales = size_t(T) * (group ? d / group : 1) * 4;
  const NormRows out[4] = {{residual_out, size_t(ldro) * 2, w2}, {y, size_t(ldy) * 2, w2}, {q, size_t(ldq), size_t(d)},
                           {q ? q_scales : nullptr, 0, n_scales}};
  for (int i = 0; i < 4; ++i) {
    const int rows = i == 3 ? 1 : T;
    if (rows_overlap(out[i].p, out[i].ld, out[i].width, rows, weight, 0, w2, 1)) return LORA_ERR_INVALID_ARG;
    for (int k = 0; k < 2; ++k)
      if (i == 3 ? rows_overlap(out[i].p, 0, n_scales, 1, in[k].p, in[k].ld, in[k].width, T) : clash(out[i], in[k], T))
        return LORA_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (rows_overlap(out[i].p, out[i].ld, out[i].width, rows, out[k].p, out[k].ld, out[k].width, T))
        return LORA_ERR_INVALID_ARG;
  }
  int n_dev = 0;
  if (cuda_status(cudaGetDeviceCount(&n_dev)) != LORA_OK) return LORA_ERR_CUDA;
  if (device < 0 || device >= n_dev) return LORA_ERR_INVALID_ARG;

  NormArgs a;
  a.x = static_cast<const uint8_t *>(x);
  a.res = static_cast<const uint8_t *>(residual);
  a.weight = static_cast<const uint8_t *>(weight);
  a.sum = static_cast<uint8_t *>(residual_out);
  a.y = static_cast<uint8_t *>(y);
  a.q = static_cast<uint8_t *>(q);
  a.scales = q_scales;
  a.ldx = 2ll * ldx;
  a.ldr = 2ll * ldr;
  a.lds = 2ll * ldro;
  a.ldy = 2ll * ldy;
  a.ldq = ldq;
  a.eps = eps;
  a.group = group;
  for (a.log2_vecs = 0; group > 8 << a.log2_vecs;) ++a.log2_vecs;
  a.T = T;
  a.d = d;
  const int nv = d / 8;
  DeviceGuard g(device);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (nv <= 32) {  // rows share a warp
    a.tpr = 2;
    while (a.tpr < nv) a.tpr *= 2;
    return launch_norm<1>(a, 256 / a.tpr, st);
  }
  int n_sm = 0;
  if (cuda_status(cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, device)) != LORA_OK) return LORA_ERR_CUDA;
  const int vpt = T > 4 * n_sm || nv > 2 * kNormMaxThreads ? 4 : 2;
  a.tpr = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
  return vpt == 4 ? launch_norm<4>(a, 1, st) : launch_norm<2>(a, 1, st);
}

}  // extern "C"
