// sv_kv8_attention_64_exact.cu -- the attention kernels over the 8-bit cache for 64 dimensions, weights in four parts.
#include "sv_kv8_attention.cuh"

namespace sv {
SV_KV8_ATTENTION_INSTANTIATE(64, 4)
}
