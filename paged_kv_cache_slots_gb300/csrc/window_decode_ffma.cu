// Launchers of the windowed decode kernel on the CUDA cores (decode_ffma.cuh): f32
// caches, and f16 and bf16 ones whose block size the tensor cores do not take.
#include "decode_ffma.cuh"

namespace pkv {

namespace {

template <int DT, int D>
cudaError_t launch_g(const WindowArgs& a, cudaStream_t stream) {
    const CUtensorMap none{};
    switch (a.num_q_heads / a.num_kv_heads) {
        case 1: return launch_window<FfmaPolicy<DT, D, 1>>(a, none, none, stream);
        case 2: return launch_window<FfmaPolicy<DT, D, 2>>(a, none, none, stream);
        case 4: return launch_window<FfmaPolicy<DT, D, 4>>(a, none, none, stream);
        case 8: return launch_window<FfmaPolicy<DT, D, 8>>(a, none, none, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <int DT>
cudaError_t launch_d(const WindowArgs& a, cudaStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch_g<DT, 64>(a, stream);
        case 128: return launch_g<DT, 128>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_window_decode_ffma(const WindowArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case kF32: return launch_d<kF32>(a, stream);
        case kF16: return launch_d<kF16>(a, stream);
        case kBF16: return launch_d<kBF16>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
