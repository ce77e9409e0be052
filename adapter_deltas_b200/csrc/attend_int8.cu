// attend_int8.cu -- the attention kernels over int8 caches (attend.cuh).
#include "attend.cuh"

namespace lora {

Variant attend_variant_int8(int dim) { return variant_of<LORA_KV_INT8>(dim); }

}  // namespace lora
