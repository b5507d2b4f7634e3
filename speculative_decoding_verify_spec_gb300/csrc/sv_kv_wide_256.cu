// sv_kv_wide_256.cu -- the attention kernel for many rows and 256 dimensions.
#include "sv_kv_wide.cuh"

namespace sv {
template <int D, bool kExact>
cudaError_t launch_wide_of(const AttArgs &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide_of<256, false>(const AttArgs &a, int grid, cudaStream_t s) {
    return launch_wide<256, false>(a, grid, s);
}
}  // namespace sv
