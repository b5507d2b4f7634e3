// sv_kv_attention_64_exact.cu -- the attention kernels for 64 dimensions, queries in two parts.
#include "sv_kv_attention.cuh"

namespace sv {
SV_KV_ATTENTION_INSTANTIATE(64, true)
}  // namespace sv
