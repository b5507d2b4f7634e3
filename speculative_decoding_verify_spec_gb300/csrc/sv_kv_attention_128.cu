// sv_kv_attention_128.cu -- the attention kernels for 128 dimensions.
#include "sv_kv_attention.cuh"

namespace sv {
SV_KV_ATTENTION_INSTANTIATE(128, false)
}  // namespace sv
