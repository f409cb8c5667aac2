// Launchers of the windowed tcgen05 kernel (window_prefill_tc.cuh) for f16 and bf16 caches, and its plan.
#include "window_prefill_tc.cuh"

namespace pkv {

namespace {

// The items' tiles of tokens: for x = 0, 1, ... over the sequences in order, eight
// words: sequence, its first token (of all), tokens, position of the first, cached
// tokens.  tile_cum[num_seqs] gets their number.  One block; flags and leaves out a
// sequence with more new tokens than cached ones, or a length past its table.
__global__ void __launch_bounds__(1024) window_prefill_plan_kernel(const PrefillArgs a) {
    __shared__ int32_t warp_sum[32];
    pdl_allow_next();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    int carry = 0;
    for (int base = 0; base < a.num_seqs; base += 1024) {
        const int s = base + tid;
        int n = 0, c = 0, start = 0, v = 0;
        if (s < a.num_seqs) {
            start = a.query_start[s];
            n = a.query_start[s + 1] - start;
            c = a.context_lens[s];
            if (n < 0 || n > c || c > a.max_blocks * a.block_size || start < 0 || start > a.num_tokens - n) {
                raise_flag(a.status, kFlagBadContext);
                n = 0;
            }
            v = (n + a.tile_tokens - 1) / a.tile_tokens;
        }
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[wid] = x;
        __syncthreads();
        if (wid == 0) {
            int w = warp_sum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += y;
            }
            warp_sum[lane] = w;
        }
        __syncthreads();
        int at = carry + (wid > 0 ? warp_sum[wid - 1] : 0) + x - v;
        carry += warp_sum[31];
        for (int q = 0; q < v && at < a.grid_tiles; ++q, ++at) {
            int4* d = reinterpret_cast<int4*>(a.tiles) + 2 * static_cast<int64_t>(at);
            d[0] = make_int4(s, start + q * a.tile_tokens, min(a.tile_tokens, n - q * a.tile_tokens), c - n + q * a.tile_tokens);
            d[1] = make_int4(c, 0, 0, 0);
        }
        __syncthreads();
    }
    if (tid == 0) a.tile_cum[a.num_seqs] = min(carry, a.grid_tiles);
}

template <int DT>
cudaError_t launch_tc_t(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int ctas,
                        cudaStream_t stream) {
    const bool two = a.out_dtype == kF32;
    if (a.head_dim == 64)
        return two ? launch_tc_g<DT, 64, true>(a, tmq, tmk, tmv, ctas, stream)
                   : launch_tc_g<DT, 64, false>(a, tmq, tmk, tmv, ctas, stream);
    if (a.head_dim == 128)
        return two ? launch_tc_g<DT, 128, true>(a, tmq, tmk, tmv, ctas, stream)
                   : launch_tc_g<DT, 128, false>(a, tmq, tmk, tmv, ctas, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

int window_prefill_tc_smem_bytes(int head_dim) {
    return head_dim == 128 ? static_cast<int>(Layout<128, false>::kBars + sizeof(Bars<Layout<128, false>::kStages>)) + 1024
                           : static_cast<int>(Layout<64, false>::kBars + sizeof(Bars<Layout<64, false>::kStages>)) + 1024;
}

cudaError_t launch_window_prefill_tc(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk,
                                     const CUtensorMap& tmv, int num_sms, cudaStream_t stream) {
    const cudaError_t e = launch_kernel(window_prefill_plan_kernel, dim3(1), dim3(1024), 0, stream, a.pdl != 0, a);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(a.grid_tiles) * a.num_kv_heads;
    const int ctas = static_cast<int>(items < num_sms ? items : num_sms);
    if (a.kv_dtype == kFP8) return launch_window_prefill_tc_fp8(a, tmq, ctas, stream);
    if (a.dtype == kBF16) return launch_tc_t<kBF16>(a, tmq, tmk, tmv, ctas, stream);
    if (a.dtype == kF16) return launch_tc_t<kF16>(a, tmq, tmk, tmv, ctas, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
