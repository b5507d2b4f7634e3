// sv_kv_attention_64.cu -- the attention kernels for 64 dimensions.
#include "sv_kv_attention.cuh"

namespace sv {
SV_KV_ATTENTION_INSTANTIATE(64, false)
}  // namespace sv
