// sv_kv_attention_128_exact.cu -- the attention kernels for 128 dimensions, queries in two parts.
#include "sv_kv_attention.cuh"

namespace sv {
SV_KV_ATTENTION_INSTANTIATE(128, true)
}  // namespace sv
