// Launchers of the warp-level tensor-core decode kernel (decode_mma.cuh).
#include "decode_mma.cuh"

namespace pkv {

// Launches of up to 12 warps (the default is 9) use the instantiation built
// for 384 threads, whose register budget (168 a thread) holds the consumer
// state and the merge of split pairs without spilling.
template <int DT, int D>
static cudaError_t launch_mma_t(const DecodeArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                cudaStream_t stream) {
    if (32 * (1 + a.consumer_warps) <= 32 * 12) return launch_partial<MmaPolicy<DT, D, 32 * 12>>(a, tmk, tmv, stream);
    return launch_partial<MmaPolicy<DT, D>>(a, tmk, tmv, stream);
}

cudaError_t launch_decode_mma(const DecodeArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                              cudaStream_t stream) {
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
