// The streaming GEMM's launches with adapters.
#include "q4_gemm_stream_kernel.h"

namespace q4 {

hipError_t launch_gemm_adapters(const q4_matrix* h, const uint16_t* x, const uint16_t* bias, uint16_t* out, int M,
                                bool bf16, int waves, int workers, float* partials, uint32_t* counters,
                                const q4dev::AdapterArgs& ad, hipStream_t stream)
{
    GemmAdArgs p;
    if (!gemm_args(p, h, x, bias, out, M, waves, workers, partials, counters)) return hipErrorInvalidValue;
    p.ad = ad;
    return launch_any(h, p, bf16, waves, stream);
}

}  // namespace q4
