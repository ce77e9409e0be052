// attend.cu -- launches of the attention over the paged cache: which variant,
// how many warps and stages, and where the workspace's parts lie (attend.cuh
// has the kernel and its reasons).
#include "attend.cuh"

namespace lora {

namespace {

Variant variant_of(int type, int dim) {
  return type == LORA_KV_BF16   ? attend_variant_bf16(dim)
         : type == LORA_KV_E4M3 ? attend_variant_e4m3(dim)
                                : attend_variant_int8(dim);
}

// Warps and stages: the most warps that leave each 2 stages; their first pieces (state_bytes each) stay in shared memory where
// that costs no warp.
struct Geometry {
  int warps, stages, first;  // first: its offset in dynamic shared memory (0: in the workspace)
  int smem;
};
Geometry geometry(int most, int stage_bytes, int state_bytes) {
  const int room = kAttSmem - kAttStatic, least = 2;
  Geometry g;
  g.warps = room / (least * stage_bytes);
  g.warps = g.warps > most ? most : g.warps;
  const int keep = g.warps * state_bytes;
  const bool fits = room - keep >= least * stage_bytes * g.warps;
  g.stages = (room - (fits ? keep : 0)) / (g.warps * stage_bytes);
  g.stages = g.stages > kAttMaxStages ? kAttMaxStages : g.stages;
  g.first = fits ? g.warps * g.stages * stage_bytes : 0;
  g.smem = g.warps * g.stages * stage_bytes + (fits ? keep : 0);
  return g;
}

// A number for each launch of the process, spread over 48 bits so that what a
// workspace holds from another use does not look like one.
unsigned long long next_tag() {
  static std::atomic<uint64_t> n{1};
  return n.fetch_add(1) * 0x9e3779b97f4aull % ((1ull << 48) - 2) + 1;
}

int group_of(const lora_kv *kv, int n_heads) { return n_heads / kv->heads; }

}  // namespace

int attend_setup(lora_kv *kv) {
  const Variant v = variant_of(kv->type, kv->dim);
  for (AttendKernel k : v.kernel) {
    const int rc = cuda_status(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttSmem - kAttStatic));
    if (rc != LORA_OK) return rc;
  }
  return LORA_OK;
}

size_t attend_workspace_bytes(const lora_kv *kv, int n_heads) {
  const int group = group_of(kv, n_heads);
  const size_t state = size_t(state_floats(group > 16 ? 16 : group, kv->dim)) * 4;
  return align256(size_t(kv->n_sm) * 8) + size_t(kv->n_sm) * (2 + kAttMaxWarps) * state;
}

int launch_attend(const lora_kv *kv, int layer, const KvSeqs &s, const AttendCall &c, cudaStream_t st) {
  const Variant v = variant_of(kv->type, kv->dim);
  AttendArgs a;
  a.q = static_cast<const uint8_t *>(c.q);
  a.out = static_cast<uint8_t *>(c.out);
  a.ldq = 2ll * c.ldq;
  a.ldo = 2ll * c.ldo;
  a.lse = c.lse;
  a.sinks = c.sinks;
  a.n_heads = c.n_heads;
  a.group = group_of(kv, c.n_heads);
  const bool wide = a.group > 8;
  const int unit_rows = wide ? 16 : 8;
  a.rows = a.group < unit_rows ? a.group : unit_rows;
  a.head_groups = (a.group + unit_rows - 1) / unit_rows;
  a.units = kv->heads * a.head_groups;
  a.scale2 = c.scale * 1.44269504f;
  a.window = c.window;
  a.stall = c.stall;
  a.wait_ns = wait_limit_ns();
  const size_t floats = state_floats(a.rows, kv->dim);
  const Geometry g = geometry(v.warps[wide], v.tt * kv_tile_bytes(kv->type, kv->dim), int(floats * 4));
  a.n_stages = g.stages;
  a.first_in_smem = g.first;
  uint8_t *ws = static_cast<uint8_t *>(c.ws);
  a.done = reinterpret_cast<unsigned long long *>(ws);
  a.tag = next_tag();
  a.part = reinterpret_cast<float *>(ws + align256(size_t(kv->n_sm) * 8));
  a.first = a.part + size_t(kv->n_sm) * 2 * floats;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kv->n_sm);
  cfg.blockDim = dim3(g.warps * 32);
  cfg.dynamicSmemBytes = g.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int rc = cuda_status(cudaLaunchKernelEx(&cfg, v.kernel[wide], kv->view(layer), s, a));
  if (rc == LORA_OK) g_launches.fetch_add(1);
  return rc;
}

}  // namespace lora
