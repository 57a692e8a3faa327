// The skinny kernel's launches with adapters.
#include "q4_gemv_kernel.h"

namespace q4 {

hipError_t launch_gemv_adapters(const q4_matrix* h, const uint16_t* x, const uint16_t* bias, uint16_t* out, int M,
                                int col_tiles, int splits, bool gather_x, bool bf16, float* partials,
                                uint32_t* counters, const q4dev::AdapterArgs& ad, hipStream_t stream)
{
    GemvAdArgs p;
    if (!gemv_args(p, h, x, bias, out, M, splits, gather_x, partials, counters)) return hipErrorInvalidValue;
    p.ad = ad;
    return launch_any(h, p, col_tiles, splits, gather_x, bf16, stream);
}

}  // namespace q4
