// sv_kv8_attention_128.cu -- the attention kernels over the 8-bit cache for 128 dimensions, weights in three parts.
#include "sv_kv8_attention.cuh"

namespace sv {
SV_KV8_ATTENTION_INSTANTIATE(128, 3)
}
