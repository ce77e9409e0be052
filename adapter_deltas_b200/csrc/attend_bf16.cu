// attend_bf16.cu -- the attention kernels over bf16 caches (attend.cuh).
#include "attend.cuh"

namespace lora {

Variant attend_variant_bf16(int dim) { return variant_of<LORA_KV_BF16>(dim); }

}  // namespace lora
