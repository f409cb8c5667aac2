// Launchers of the warp-MMA kernel of multi-token queries with a sliding window over
// an E4M3 cache (prefill_mma.cuh).
#include "prefill_mma.cuh"

namespace pkv {

cudaError_t launch_window_prefill(const PrefillArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                  cudaStream_t stream) {
    if (a.kv_dtype != kFP8 || a.head_dim != 128) return cudaErrorInvalidValue;
    if (a.dtype == kF16) return launch_prefill_t<kF16, 128, true, true>(a, tmk, tmv, stream);
    if (a.dtype == kBF16) return launch_prefill_t<kBF16, 128, true, true>(a, tmk, tmv, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
