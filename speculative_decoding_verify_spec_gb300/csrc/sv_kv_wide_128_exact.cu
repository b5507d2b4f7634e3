// sv_kv_wide_128_exact.cu -- the attention kernel for many rows and 128 dimensions, queries in two parts.
#include "sv_kv_wide.cuh"

namespace sv {
template <int D, bool kExact>
cudaError_t launch_wide_of(const AttArgs &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide_of<128, true>(const AttArgs &a, int grid, cudaStream_t s) {
    return launch_wide<128, true>(a, grid, s);
}
}  // namespace sv
