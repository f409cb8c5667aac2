// Shared-prefix attention over f16 caches (shared_prefix_kernel.cuh).
#include "decode_mma.cuh"
#include "shared_prefix_kernel.cuh"

namespace pkv {

cudaError_t launch_attend_f16(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmk,
                               const CUtensorMap& tmv, cudaStream_t stream) {
    if (d.head_dim == 64) return launch_attend_t<MmaPolicy<kF16, 64, parts_threads(false)>, kF16, 64, false>(a, d, tmk, tmv, stream);
    return launch_attend_t<MmaPolicy<kF16, 128, parts_threads(false)>, kF16, 128, false>(a, d, tmk, tmv, stream);
}

int prefix_static_smem_bytes() { return static_cast<int>(sizeof(Bars)) + 64; }

int prefix_smem_bytes(int head_dim, bool fp8) {
    const uint32_t off = fp8 ? Shape<128, true>::kBytes : head_dim == 64 ? Shape<64, false>::kBytes : Shape<128, false>::kBytes;
    return static_cast<int>(off + 1024);
}

}  // namespace pkv
