// sv_kv8_wide_128.cu -- the attention kernels over the 8-bit cache for many rows and 128 dimensions.
#include "sv_kv8_wide.cuh"

namespace sv {
template <>
cudaError_t launch_wide8_of<128, 2>(const Att8Args &a, int grid, cudaStream_t s) {
    return launch_wide8<128, 2>(a, grid, s);
}
template <>
cudaError_t launch_wide8_of<128, 3>(const Att8Args &a, int grid, cudaStream_t s) {
    return launch_wide8<128, 3>(a, grid, s);
}
}  // namespace sv
