// Launchers of the windowed tcgen05 kernel (window_prefill_tc.cuh) for E4M3 caches.
#include "window_prefill_tc.cuh"

namespace pkv {

cudaError_t launch_window_prefill_tc_fp8(const PrefillArgs& a, const CUtensorMap& tmq, int ctas, cudaStream_t stream) {
    const CUtensorMap none{};
    if (a.head_dim != 128) return cudaErrorInvalidValue;
    const bool two = a.out_dtype == kF32;
    if (a.dtype == kF16)
        return two ? launch_tc_g<kF16, 128, true, true>(a, tmq, none, none, ctas, stream)
                   : launch_tc_g<kF16, 128, false, true>(a, tmq, none, none, ctas, stream);
    if (a.dtype == kBF16)
        return two ? launch_tc_g<kBF16, 128, true, true>(a, tmq, none, none, ctas, stream)
                   : launch_tc_g<kBF16, 128, false, true>(a, tmq, none, none, ctas, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
