// Launcher of the decode kernels' variant that attends to what follows a
// shared prefix (see shared_prefix.cu): partials only, leading table entries
// skipped.  One block size is built (up to 12 warps, the usual launch).
#include "decode_fp8.cuh"
#include "decode_mma.cuh"
#include "shared_prefix.cuh"

namespace pkv {

cudaError_t launch_decode_tails(const DecodeArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                cudaStream_t stream) {
    constexpr int kT = 32 * 12;
    if (a.kv_dtype == kFP8) {
        if (a.head_dim != 128) return cudaErrorInvalidValue;
        if (a.dtype == kF16) return launch_partial<MmaFp8Policy<kF16, 128, false, kT>, true>(a, tmk, tmv, stream);
        if (a.num_q_heads / a.num_kv_heads <= 4)
            return launch_partial<MmaFp8Policy<kBF16, 128, true, kT>, true>(a, tmk, tmv, stream);
        return launch_partial<MmaFp8Policy<kBF16, 128, false, kT>, true>(a, tmk, tmv, stream);
    }
    if (a.dtype == kF16) {
        if (a.head_dim == 64) return launch_partial<MmaPolicy<kF16, 64, kT>, true>(a, tmk, tmv, stream);
        if (a.head_dim == 128) return launch_partial<MmaPolicy<kF16, 128, kT>, true>(a, tmk, tmv, stream);
    } else if (a.dtype == kBF16) {
        if (a.head_dim == 64) return launch_partial<MmaPolicy<kBF16, 64, kT>, true>(a, tmk, tmv, stream);
        if (a.head_dim == 128) return launch_partial<MmaPolicy<kBF16, 128, kT>, true>(a, tmk, tmv, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pkv
