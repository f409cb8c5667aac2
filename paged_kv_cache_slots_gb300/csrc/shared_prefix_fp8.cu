// Shared-prefix attention over E4M3 caches (shared_prefix_kernel.cuh).
#include "decode_fp8.cuh"
#include "shared_prefix_kernel.cuh"

namespace pkv {

cudaError_t launch_attend_fp8(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmk,
                              const CUtensorMap& tmv, cudaStream_t stream) {
    constexpr int kT = parts_threads(true);
    if (d.dtype == kF16) return launch_attend_t<MmaFp8Policy<kF16, 128, false, kT>, kF16, 128, true>(a, d, tmk, tmv, stream);
    if (d.num_q_heads / d.num_kv_heads <= 4)
        return launch_attend_t<MmaFp8Policy<kBF16, 128, true, kT>, kBF16, 128, true>(a, d, tmk, tmv, stream);
    return launch_attend_t<MmaFp8Policy<kBF16, 128, false, kT>, kBF16, 128, true>(a, d, tmk, tmv, stream);
}

}  // namespace pkv
