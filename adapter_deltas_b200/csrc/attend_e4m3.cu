// attend_e4m3.cu -- the attention kernels over e4m3 caches (attend.cuh).
#include "attend.cuh"

namespace lora {

Variant attend_variant_e4m3(int dim) { return variant_of<LORA_KV_E4M3>(dim); }

}  // namespace lora
