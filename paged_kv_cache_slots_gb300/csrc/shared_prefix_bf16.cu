// Shared-prefix attention over bf16 caches (shared_prefix_kernel.cuh).
#include "decode_mma.cuh"
#include "shared_prefix_kernel.cuh"

namespace pkv {

cudaError_t launch_attend_bf16(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmk,
                               const CUtensorMap& tmv, cudaStream_t stream) {
    if (d.head_dim == 64) return launch_attend_t<MmaPolicy<kBF16, 64, parts_threads(false)>, kBF16, 64, false>(a, d, tmk, tmv, stream);
    return launch_attend_t<MmaPolicy<kBF16, 128, parts_threads(false)>, kBF16, 128, false>(a, d, tmk, tmv, stream);
}

}  // namespace pkv
