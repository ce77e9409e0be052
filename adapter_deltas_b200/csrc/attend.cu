// attend.cu -- attention of one new token per sequence over the paged cache.
//
// For query head h of sequence s, with key head g = h / (n_heads / heads) and
// positions j in [max(0, len - window), len):
//     s_j = scale * q . k_j,   out = sum_j e^(s_j) v_j / (sum_j e^(s_j) + e^sink),
// the sums held in fp32 with a running maximum.
#include "kv.cuh"

namespace lora {

struct AttendArgs {
  const uint8_t *q;
  uint8_t *out;
  long long ldq, ldo;
  float *lse;
  const float *sinks;
  int n_heads;
  float scale;
  int window;
};

// One warp per (sequence, query head): a plain pass over the tokens.
template <int TYPE>
__global__ void __launch_bounds__(128) attend_kernel(KvView kv, KvSeqs s, AttendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= (long long)s.n * a.n_heads) return;
  const int seq = (int)(id / a.n_heads), head = (int)(id % a.n_heads), kvh = head / (a.n_heads / kv.heads);
  const int len = s.lens[seq];
  if (len < 0 || len > ((long long)s.max_pages << kv.log2_page)) {
    if (len != -1) set_status(kv.status, LORA_ERR_BAD_ID);
    return;
  }
  const int n8 = kv.dim / 8;
  const bool on = lane < n8;  // 8 elements per lane
  float q[8] = {0}, o[8] = {0}, m = -INFINITY, l = 0.f;
  if (on) unpack8(*reinterpret_cast<const uint4 *>(a.q + seq * a.ldq + (head * kv.dim + lane * 8) * 2), q);
  const int first = a.window && len > a.window ? len - a.window : 0;
  for (int j = first; j < len; ++j) {
    const int page = s.table[(long long)seq * s.max_pages + (j >> kv.log2_page)];
    const long long at = kv_tile_offset(kv, page, j);
    if (at < 0) {
      set_status(kv.status, LORA_ERR_BAD_ID);
      continue;
    }
    constexpr int ES = kv_elt(TYPE);
    const uint8_t *t = kv.base + at + kvh * kv_head_stride(kv);
    const int row = j & 15, rb = kv.dim * ES, b = lane * 8 * ES;
    float k[8] = {0}, v[8] = {0}, ks = 1.f, vs = 1.f;
    if (on) {
      const uint8_t *pk = t + row * rb + kv_chunk(b / 16, row, rb / 16) * 16 + b % 16, *pv = pk + 16 * rb;
      if (TYPE == LORA_KV_BF16) {
        unpack8(*reinterpret_cast<const uint4 *>(pk), k);
        unpack8(*reinterpret_cast<const uint4 *>(pv), v);
      } else {
        const uint2 ck = *reinterpret_cast<const uint2 *>(pk), cv = *reinterpret_cast<const uint2 *>(pv);
        decode4<TYPE>(ck.x, k);
        decode4<TYPE>(ck.y, k + 4);
        decode4<TYPE>(cv.x, v);
        decode4<TYPE>(cv.y, v + 4);
      }
    }
    if (TYPE != LORA_KV_BF16) {
      const float *sc = reinterpret_cast<const float *>(t + 32 * rb);
      ks = sc[row];
      vs = sc[16 + row];
    }
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) dot = fmaf(q[e], k[e], dot);
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
    const float sc = dot * ks * a.scale, mn = fmaxf(m, sc);
    const float base = mn == -INFINITY ? 0.f : mn, alpha = expf(m - base), p = expf(sc - base);
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(p * vs, v[e], o[e] * alpha);
    m = mn;
  }
  if (a.sinks) {
    const float sink = a.sinks[head], mn = fmaxf(m, sink), base = mn == -INFINITY ? 0.f : mn;
    const float alpha = expf(m - base);
    l = l * alpha + expf(sink - base);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= alpha;
    m = mn;
  }
  const float inv = len > 0 || l > 0.f ? 1.f / l : 0.f;
  if (on) {
    uint4 u = make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                         pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
    *reinterpret_cast<uint4 *>(a.out + seq * a.ldo + (head * kv.dim + lane * 8) * 2) = u;
  }
  if (a.lse && lane == 0) a.lse[(long long)seq * a.n_heads + head] = (m == -INFINITY ? 0.f : m) + logf(l);
}

int attend_setup(lora_kv *) { return LORA_OK; }
size_t attend_workspace_bytes(const lora_kv *, int) { return 256; }

int launch_attend(const lora_kv *kv, int layer, const KvSeqs &s, const AttendCall &c, cudaStream_t st) {
  AttendArgs a;
  a.q = static_cast<const uint8_t *>(c.q);
  a.out = static_cast<uint8_t *>(c.out);
  a.ldq = 2ll * c.ldq;
  a.ldo = 2ll * c.ldo;
  a.lse = c.lse;
  a.sinks = c.sinks;
  a.n_heads = c.n_heads;
  a.scale = c.scale;
  a.window = c.window;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)s.n * c.n_heads + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = kv->type == LORA_KV_BF16   ? attend_kernel<LORA_KV_BF16>
                : kv->type == LORA_KV_E4M3 ? attend_kernel<LORA_KV_E4M3>
                                           : attend_kernel<LORA_KV_INT8>;
  const int rc = cuda_status(cudaLaunchKernelEx(&cfg, kernel, kv->view(layer), s, a));
  if (rc == LORA_OK) g_launches.fetch_add(1);
  return rc;
}

}  // namespace lora
