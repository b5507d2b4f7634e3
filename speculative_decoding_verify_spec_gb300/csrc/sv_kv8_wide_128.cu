// sv_kv8_wide_128.cu -- the attention kernel over the 8-bit cache for many rows and 128 dimensions.
#include "sv_kv8_wide.cuh"

namespace sv {
template <>
cudaError_t launch_wide8_of<128>(const Att8Args &a, int grid, cudaStream_t s) {
    return launch_wide8<128>(a, grid, s);
}
}  // namespace sv
