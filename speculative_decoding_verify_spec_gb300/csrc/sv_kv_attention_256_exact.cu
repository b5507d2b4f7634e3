// sv_kv_attention_256_exact.cu -- the attention kernels for 256 dimensions, queries in two parts.
#include "sv_kv_attention.cuh"

namespace sv {
SV_KV_ATTENTION_INSTANTIATE(256, true)
}  // namespace sv
