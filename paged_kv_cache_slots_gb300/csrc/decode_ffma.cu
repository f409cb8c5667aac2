// Launchers of the CUDA-core decode kernel (decode_ffma.cuh).
#include "decode_ffma.cuh"

namespace pkv {

template <int DT, int D, int G>
static cudaError_t launch_ffma_t(const DecodeArgs& a, cudaStream_t stream) {
    CUtensorMap none{};
    return launch_partial<FfmaPolicy<DT, D, G>>(a, none, none, stream);
}

template <int DT, int D>
static cudaError_t launch_ffma_g(const DecodeArgs& a, cudaStream_t stream) {
    switch (a.num_q_heads / a.num_kv_heads) {
        case 1: return launch_ffma_t<DT, D, 1>(a, stream);
        case 2: return launch_ffma_t<DT, D, 2>(a, stream);
        case 4: return launch_ffma_t<DT, D, 4>(a, stream);
        case 8: return launch_ffma_t<DT, D, 8>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <int DT>
static cudaError_t launch_ffma_d(const DecodeArgs& a, cudaStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch_ffma_g<DT, 64>(a, stream);
        case 128: return launch_ffma_g<DT, 128>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_decode_ffma(const DecodeArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case kF32: return launch_ffma_d<kF32>(a, stream);
        case kF16: return launch_ffma_d<kF16>(a, stream);
        case kBF16: return launch_ffma_d<kBF16>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
