// Launchers of the windowed decode kernel for f16 and bf16 caches (decode_mma.cuh)
// and for E4M3 ones (decode_fp8.cuh); the same variants as without a window.  Bound:
// HBM, of what is in sight alone.  256 sequences under a window of 2,048, 8 KV heads of
// 128 (2.03 GB): 296 us, the rate of a copy; 32 under one of 4,096 (497 MB): 79.5 us,
// 92 % of it; 48 over an E4M3 cache under one of 2,047 (178 MB): 38.8 us, 67 %.
#include "decode_fp8.cuh"
#include "decode_mma.cuh"

namespace pkv {

namespace {

template <int DT, int D>
cudaError_t launch_mma_t(const WindowArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t stream) {
    if (32 * (1 + a.consumer_warps) <= 32 * 12) return launch_window<MmaPolicy<DT, D, 32 * 12>>(a, tmk, tmv, stream);
    return launch_window<MmaPolicy<DT, D>>(a, tmk, tmv, stream);
}

cudaError_t launch_fp8(const WindowArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t stream) {
    if (a.head_dim != 128) return cudaErrorInvalidValue;
    const int G = a.num_q_heads / a.num_kv_heads;
    if (a.dtype == kF16) return launch_window<MmaFp8Policy<kF16, 128>>(a, tmk, tmv, stream);
    if (a.dtype == kBF16 && G <= 4) {
        if (32 * (1 + a.consumer_warps) <= 32 * 12)
            return launch_window<MmaFp8Policy<kBF16, 128, true, 32 * 12>>(a, tmk, tmv, stream);
        return launch_window<MmaFp8Policy<kBF16, 128, true>>(a, tmk, tmv, stream);
    }
    if (a.dtype == kBF16) return launch_window<MmaFp8Policy<kBF16, 128>>(a, tmk, tmv, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_window_decode_mma(const WindowArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                     cudaStream_t stream) {
    if (a.kv_dtype == kFP8) return launch_fp8(a, tmk, tmv, stream);
    if (a.dtype == kF16) {
        if (a.head_dim == 64) return launch_mma_t<kF16, 64>(a, tmk, tmv, stream);
        if (a.head_dim == 128) return launch_mma_t<kF16, 128>(a, tmk, tmv, stream);
    } else if (a.dtype == kBF16) {
        if (a.head_dim == 64) return launch_mma_t<kBF16, 64>(a, tmk, tmv, stream);
        if (a.head_dim == 128) return launch_mma_t<kBF16, 128>(a, tmk, tmv, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pkv
