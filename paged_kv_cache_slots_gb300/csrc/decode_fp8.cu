// Launcher of the E4M3 decode kernel (decode_fp8.cuh).
#include "decode_fp8.cuh"

namespace pkv {

cudaError_t launch_decode_fp8(const DecodeArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                              cudaStream_t stream) {
    if (a.kv_dtype != kFP8 || a.head_dim != 128) return cudaErrorInvalidValue;
    const int G = a.num_q_heads / a.num_kv_heads;
    if (a.dtype == kF16) return launch_partial<MmaFp8Policy<kF16, 128>>(a, tmk, tmv, stream);
    if (a.dtype == kBF16 && G <= 4) {
        if (32 * (1 + a.consumer_warps) <= 32 * 12)
            return launch_partial<MmaFp8Policy<kBF16, 128, true, 32 * 12>>(a, tmk, tmv, stream);
        return launch_partial<MmaFp8Policy<kBF16, 128, true>>(a, tmk, tmv, stream);
    }
    if (a.dtype == kBF16) return launch_partial<MmaFp8Policy<kBF16, 128>>(a, tmk, tmv, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
