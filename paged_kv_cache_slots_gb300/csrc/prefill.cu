// Multi-token queries over the paged cache (chunked prefill: "Batching and
// Scheduling", Example 5; "vLLM Architecture and Installation", Example 5).
//
// A step gives sequence s n_s = query_start[s+1] - query_start[s] new tokens
// (1 for a decoding request, a chunk of the prompt for a prefilling one),
// already appended, so its cache holds context_lens[s] tokens and new token i
// sits at position p_i = context_lens[s] - n_s + i.  Token i attends to the
// cached tokens at positions 0 .. p_i (causal), read through the block table.
//
// Work split: one CTA per (tile of 16 new tokens of one sequence, KV head).
// Warp 0 streams that head's K and V tiles of the blocks the tile needs
// (positions up to the tile's last p_i) into a ring of shared-memory stages
// with TMA (128-byte swizzle, as the decode kernel); warp 1 + w computes query
// head h*G + w for the 16 tokens, in the usual flash-attention register layout:
//   S[16 tok x 16 keys] = Q[16 x D] . K^T     (m16n8k16, Q in registers, K by ldmatrix)
//   causal mask, online softmax per row (fp32, base 2)
//   O[16 x D] += P[16 x 16] . V[16 x D]       (P from the S registers as the A
//                                             operand, high + low halves; V by ldmatrix.trans)
// The tile index -> (sequence, tile) map comes from a small plan kernel
// (prefix of tiles per sequence in the workspace).
#include "prefill_mma.cuh"

namespace pkv {

namespace {

// cum[s] = sum_{s' < s} ceil(n_s' / tile_tokens); cum[B] = tiles.  One block; flags
// a chunk longer than its context or a decreasing query_start.
__global__ void __launch_bounds__(1024) prefill_plan_kernel(const PrefillArgs a) {
    pdl_allow_next();
    pdl_wait();
    __shared__ int32_t warp_sum[32];
    __shared__ int32_t carry_s;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) carry_s = 0;
    __syncthreads();
    for (int base = 0; base < a.num_seqs; base += blockDim.x) {
        const int s = base + tid;
        int v = 0;
        if (s < a.num_seqs) {
            const int n = a.query_start[s + 1] - a.query_start[s];
            const int c = a.context_lens[s];
            if (n < 0 || n > c || c > a.max_blocks * a.block_size) raise_flag(a.status, kFlagBadContext);
            v = n > 0 && n <= c && c <= a.max_blocks * a.block_size ? (n + a.tile_tokens - 1) / a.tile_tokens : 0;
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
            const int nw = blockDim.x >> 5;
            int t = lane < nw ? warp_sum[lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += y;
            }
            warp_sum[lane] = t;
        }
        __syncthreads();
        const int before = carry_s + (wid > 0 ? warp_sum[wid - 1] : 0);
        if (s < a.num_seqs) a.tile_cum[s] = before + x - v;
        __syncthreads();
        if (tid == 0) carry_s += warp_sum[(blockDim.x >> 5) - 1];
        __syncthreads();
    }
    if (tid == 0) a.tile_cum[a.num_seqs] = carry_s;
}

// f32 q and cache: one warp per (new token, query head), the token's causal
// prefix one key at a time on the CUDA cores (lane l holds dims VD*l ..
// VD*l + VD - 1; the dot product reduced across the warp), online softmax in
// base 2.  A sequence whose chunk is longer than its context, or whose context
// exceeds its table, writes nothing (the plan kernel flags it).  kWindow: only
// the keys in sight (see prefill_mma.cuh).
template <int D, bool kWindow>
__global__ void __launch_bounds__(256) paged_prefill_f32_kernel(const PrefillArgs a) {
    constexpr int VD = D / 32;
    pdl_allow_next();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(a.num_tokens) * a.num_q_heads) return;
    const int64_t tok = row / a.num_q_heads;
    const int g = static_cast<int>(row - tok * a.num_q_heads);
    const int h = g / (a.num_q_heads / a.num_kv_heads);
    int lo = 0, hi = a.num_seqs;  // the sequence of the token: largest s with query_start[s] <= tok
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.query_start[mid] <= tok) lo = mid; else hi = mid;
    }
    const int s = lo;
    const int n = a.query_start[s + 1] - a.query_start[s];
    const int ctx = a.context_lens[s];
    if (n <= 0 || n > ctx || ctx > a.max_blocks * a.block_size) return;
    if (kWindow && tok - a.query_start[s] >= n) return;  // a row behind the last sequence
    const int pos = ctx - n + static_cast<int>(tok - a.query_start[s]);
    const float* qrow = static_cast<const float*>(a.q) + row * D + VD * lane;
    float q[VD], o[VD];
#pragma unroll
    for (int i = 0; i < VD; ++i) {
        q[i] = qrow[i] * a.scale_log2;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const float* kc = static_cast<const float*>(a.k_cache);
    const float* vc = static_cast<const float*>(a.v_cache);
    const int from = kWindow ? max(0, pos - a.window + 1) : 0;
    for (int t = kWindow && a.sinks == 0 ? from : 0; t <= pos; ++t) {
        if (kWindow && t >= a.sinks && t < from) t = from;
        int blk = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + t / a.block_size];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) raise_flag(a.status, kFlagBadBlock);
            blk = 0;
        }
        const int64_t r = (static_cast<int64_t>(blk) * a.num_kv_heads + h) * a.block_size + t % a.block_size;
        const float* k = kc + r * D + VD * lane;
        const float* v = vc + r * D + VD * lane;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < VD; ++i) x = fmaf(q[i], __ldg(k + i), x);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        const float mn = fmaxf(m, x);
        const float al = fast_exp2(m - mn);  // 0 while m is -inf
        const float p = fast_exp2(x - mn);
        l = fmaf(l, al, p);
#pragma unroll
        for (int i = 0; i < VD; ++i) o[i] = fmaf(o[i], al, p * __ldg(v + i));
        m = mn;
    }
    const float inv = 1.f / l;
    float* out = static_cast<float*>(a.out) + row * D + VD * lane;
#pragma unroll
    for (int i = 0; i < VD; ++i) out[i] = o[i] * inv;
}

template <bool kWindow>
cudaError_t launch_prefill_f32(const PrefillArgs& a, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(a.num_tokens) * a.num_q_heads;
    const int blocks = static_cast<int>((warps + 7) / 8);
    if (a.head_dim == 64) return launch_kernel(paged_prefill_f32_kernel<64, kWindow>, dim3(blocks), dim3(256), 0, stream,
                                               a.pdl != 0, a);
    if (a.head_dim == 128) return launch_kernel(paged_prefill_f32_kernel<128, kWindow>, dim3(blocks), dim3(256), 0, stream,
                                                a.pdl != 0, a);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                           cudaStream_t stream) {
    if (a.num_seqs == 0 || a.num_tokens == 0) return cudaSuccess;
    cudaError_t e = launch_kernel(prefill_plan_kernel, dim3(1), dim3(1024), 0, stream, a.pdl != 0, a);
    if (e != cudaSuccess) return e;
    if (a.window > 0) {
        if (a.dtype == kF32) return launch_prefill_f32<true>(a, stream);
        return launch_window_prefill(a, tmk, tmv, stream);
    }
    if (a.kv_dtype == kFP8) {
        if (a.head_dim != 128) return cudaErrorInvalidValue;
        if (a.dtype == kF16) return launch_prefill_t<kF16, 128, true>(a, tmk, tmv, stream);
        if (a.dtype == kBF16) return launch_prefill_t<kBF16, 128, true>(a, tmk, tmv, stream);
        return cudaErrorInvalidValue;
    }
    if (a.dtype == kF32) return launch_prefill_f32<false>(a, stream);
    if (a.tensor_cores) return launch_prefill_tc(a, tmk, tmv, stream);
    if (a.dtype == kF16) {
        if (a.head_dim == 64) return launch_prefill_t<kF16, 64>(a, tmk, tmv, stream);
        if (a.head_dim == 128) return launch_prefill_t<kF16, 128>(a, tmk, tmv, stream);
    } else if (a.dtype == kBF16) {
        if (a.head_dim == 64) return launch_prefill_t<kBF16, 64>(a, tmk, tmv, stream);
        if (a.head_dim == 128) return launch_prefill_t<kBF16, 128>(a, tmk, tmv, stream);
    }
    return cudaErrorInvalidValue;
}

// Slot of every new token: token i of sequence s at position context_lens[s] - n_s + i.
__global__ void __launch_bounds__(128) kv_slot_mapping_varlen_kernel(const PrefillArgs a, int32_t* slots) {
    pdl_allow_next();
    pdl_wait();
    const int s = blockIdx.x;
    if (s >= a.num_seqs) return;
    const int q0 = a.query_start[s], q1 = a.query_start[s + 1];
    const int n = q1 - q0, ctx = a.context_lens[s];
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int pos = ctx - n + i;
        int32_t slot = -1;
        const int j = pos >= 0 ? pos / a.block_size : -1;
        if (pos < 0 || j >= a.max_blocks) {
            raise_flag(a.status, kFlagBadContext);
        } else {
            const int blk = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + j];
            if (blk < 0 || blk >= a.num_blocks)
                raise_flag(a.status, kFlagBadBlock);
            else
                slot = blk * a.block_size + (pos - j * a.block_size);
        }
        if (q0 + i < a.num_tokens) slots[q0 + i] = slot;
    }
}

cudaError_t launch_slot_mapping_varlen(const PrefillArgs& a, int32_t* slots, cudaStream_t stream) {
    if (a.num_seqs == 0) return cudaSuccess;
    return launch_kernel(kv_slot_mapping_varlen_kernel, dim3(a.num_seqs), dim3(128), 0, stream,
                         a.pdl != 0, a, slots);
}

}  // namespace pkv
