// sv_kv_attention_256.cu -- the attention kernels for 256 dimensions.
#include "sv_kv_attention.cuh"

namespace sv {
SV_KV_ATTENTION_INSTANTIATE(256, false)
}  // namespace sv
