// Instantiations of the many-row attention kernel for a cache of 16 bits.
#include "q4_attend_tiles_kernel.h"

namespace q4 {

hipError_t launch_attend_tiles(const q4attend::Args& p, int grid, bool bf16, bool pages_of_16, hipStream_t stream)
{
    if (p.dim < 8 || p.dim > 256 || p.dim % 8 || grid < 1 || p.workers < 1) return hipErrorInvalidValue;
    if (p.sinks) {
        if (p.dim <= 64) return launch_tiles<64, true, false>(p, grid, bf16, pages_of_16, stream);
        if (p.dim <= 128) return launch_tiles<128, true, false>(p, grid, bf16, pages_of_16, stream);
        return launch_tiles<256, true, false>(p, grid, bf16, pages_of_16, stream);
    }
    if (p.dim <= 64) return launch_tiles<64, false, false>(p, grid, bf16, pages_of_16, stream);
    if (p.dim <= 128) return launch_tiles<128, false, false>(p, grid, bf16, pages_of_16, stream);
    return launch_tiles<256, false, false>(p, grid, bf16, pages_of_16, stream);
}

}  // namespace q4
