// Windowed decode for small batches and short windows (f16, bf16 and E4M3 caches):
// the same operation as paged_window_decode_kernel (decode_kernel.cuh), for calls that
// are bound by latency rather than by what they read.
//
// Work split.  A cluster of 1, 2, 4 or 8 CTAs takes one (sequence, KV head).  Its warps
// take the blocks in sight in turn: each brings its blocks of this head's K and V by
// TMA into two stages of its own, runs the tile code of the persistent kernel's
// consumers on them, and leaves its state (O, maximum, sum) in its own stage.  Each
// CTA joins its warps' states in shared memory, the cluster joins its CTAs' through
// distributed shared memory, every CTA a part of the output's elements.  So nothing
// goes through L2 but K, V, q and out, and no counter has to be kept: the persistent
// kernel's merge by the last arrival took most of a small call's time.  Bound: latency
// (table entry, TMA, tile, joins).  One sequence under a window of 1,024, 8 KV heads of
// 128, bf16: 8.0 us in a graph, the persistent kernel 35.
#include <cooperative_groups.h>

#include "decode_fp8.cuh"
#include "decode_mma.cuh"

namespace pkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxWarps = 8;
constexpr int kMaxStages = 2;  // of each warp

// Shared memory of a warp: its stages, or its state if that is larger (8 heads of 130 floats).
__host__ __device__ inline uint32_t warp_bytes(int stages, uint32_t half) {
    return stages * 2 * half < 5120u ? 5120u : stages * 2 * half;
}

template <class Policy>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) paged_window_decode_small_kernel(const WindowArgs a,
                                                                                       const __grid_constant__ CUtensorMap tmk,
                                                                                       const __grid_constant__ CUtensorMap tmv) {
    const int kStages = a.stages;
    constexpr int D = Policy::kD;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxWarps][kMaxStages];
    __shared__ int abort_flag;
    __shared__ float joined[8 * (D + 2)];  // the CTA's state: [head][O, maximum, sum]
    cg::cluster_group cluster = cg::this_cluster();
    pdl_allow_next();
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    volatile int* abort = &abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int pair = blockIdx.x / ctas;
    const int s = pair / a.num_kv_heads, h = pair - s * a.num_kv_heads;
    const int G = a.num_q_heads / a.num_kv_heads;
    const int bs = a.block_size;
    const uint32_t half = static_cast<uint32_t>(bs) * D * dtype_bytes(a.kv_dtype);
    if (tid == 0) {
        *abort = 0;
        prefetch_tensor_map(&tmk);
        prefetch_tensor_map(&tmv);
    }
    if (lane == 0) {
        for (int k = 0; k < kStages; ++k) mbar_init(&full[warp][k], 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    const int ctx = clamp_context(a, s, h == 0 && rank == 0 && tid == 0);
    const int64_t out0 = (static_cast<int64_t>(s) * a.num_q_heads + h * G) * D;
    if (ctx == 0) {  // (the whole cluster)
        if (rank == 0)
            for (int e = tid; e < G * D; e += blockDim.x) store_out(a.out, out0 + e, 0.f, a.out_dtype);
        return;
    }
    const int skip = max(0, max(0, ctx - a.window) / bs - a.sink_blocks);
    const int blocks = (ctx + bs - 1) / bs - skip;
    auto logical = [&](int j) { return j + (j >= a.sink_blocks ? skip : 0); };
    const int first = warp * ctas + rank, step = warps * ctas;
    const int mine = first < blocks ? (blocks - first + step - 1) / step : 0;
    uint8_t* stages = base + warp * warp_bytes(kStages, half);
    const uint64_t policy = policy_evict_first();
    // Row of block `k` of this warp's in the caches' tensor maps.
    auto row_of = [&](int k) {
        int blk = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + logical(first + k * step)];
        if (blk < 0 || blk >= a.num_blocks) {
            raise_flag(a.status, kFlagBadBlock);
            blk = 0;
        }
        return (blk * a.num_kv_heads + h) * bs;
    };
    auto fetch = [&](int k, int row) {  // lane 0
        const int per = 128 / dtype_bytes(a.kv_dtype), slices = D / per;
        uint8_t* kd = stages + (k % kStages) * 2 * half;
        uint64_t* bar = &full[warp][k % kStages];
        mbar_arrive_expect_tx(bar, 2 * half);
        for (int sl = 0; sl < slices; ++sl) {
            tensor_load_2d(kd + sl * (half / slices), &tmk, sl * per, row, bar, policy);
            tensor_load_2d(kd + half + sl * (half / slices), &tmv, sl * per, row, bar, policy);
        }
    };
    if (lane == 0 && mine > 0) {
        const bool second = mine > 1 && kStages > 1;
        const int r0 = row_of(0), r1 = second ? row_of(1) : 0;
        fetch(0, r0);
        if (second) fetch(1, r1);
    }
    Policy pol;
    typename Policy::State st;
    pol.begin(st, a, s, h, G);
    bool ok = true;
    int k = 0;
    for (; k < mine; ++k) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[warp][k % kStages], (k / kStages) & 1, abort, a.status));
        if (!ok) break;
        int row = 0;
        if (lane == 0 && k + kStages < mine) row = row_of(k + kStages);
        const int t0 = logical(first + k * step) * bs;
        uint8_t* kt = stages + (k % kStages) * 2 * half;
        pol.template tile<true>(st, a, kt, kt + half, 0, min(bs, ctx - t0), G, nullptr,
                                Hidden{max(a.sinks - t0, 0), min(ctx - a.window - t0, bs), lower_of(ctx, a.window)});
        __syncwarp();
        if (lane == 0 && k + kStages < mine) fetch(k + kStages, row);
    }
    if (!ok && lane == 0) {  // what was issued lands before the CTA ends (a wait gave up; bounded)
        for (int j = k; j < mine && j < k + kStages; ++j) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&full[warp][j % kStages], (j / kStages) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
    }
    float* state = reinterpret_cast<float*>(stages);  // this warp's stages hold nothing more
    pol.write_state(st, a, state, D + 2, G);
    __syncthreads();
    // The state of `n` parts (part(i): its [head][O, maximum, sum]), element (g, d): joined O, maximum and sum.
    auto join = [&](int n, auto part, int g, int d, float* o, float* m, float* l) {
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int i = 0; i < n; ++i) M = fmaxf(M, part(i)[g * (D + 2) + D]);
        for (int i = 0; i < n; ++i) {
            const float* p = part(i) + g * (D + 2);
            if (p[D + 1] == 0.f) continue;  // (no block)
            const float w = fast_exp2(p[D] - M);
            L += w * p[D + 1];
            O += w * p[d];
        }
        *o = O;
        *m = M;
        *l = L;
    };
    const int floats = static_cast<int>(warp_bytes(kStages, half)) / 4;  // between two warps' states
    auto of_warp = [&](int i) { return reinterpret_cast<const float*>(base) + static_cast<int64_t>(i) * floats; };
    if (ctas == 1) {
        for (int e = tid; e < G * D; e += blockDim.x) {
            float o, m, l;
            join(warps, of_warp, e / D, e % D, &o, &m, &l);
            store_out(a.out, out0 + e, o / l, a.out_dtype);
        }
        return;
    }
    for (int e = tid; e < G * D; e += blockDim.x) {
        const int g = e / D, d = e % D;
        float o, m, l;
        join(warps, of_warp, g, d, &o, &m, &l);
        joined[g * (D + 2) + d] = o;
        if (d == 0) {
            joined[g * (D + 2) + D] = m;
            joined[g * (D + 2) + D + 1] = l;
        }
    }
    cluster.sync();
    auto of_cta = [&](int i) { return static_cast<const float*>(cluster.map_shared_rank(joined, i)); };
    const int share = (G * D + ctas - 1) / ctas;
    for (int e = rank * share + tid; e < min(G * D, (rank + 1) * share); e += blockDim.x) {
        float o, m, l;
        join(ctas, of_cta, e / D, e % D, &o, &m, &l);
        store_out(a.out, out0 + e, o / l, a.out_dtype);
    }
    cluster.sync();  // the others have read this CTA's shared memory
}

template <class Policy>
cudaError_t launch(const WindowArgs& args, const CUtensorMap& tmk, const CUtensorMap& tmv, const SmallPlan& plan,
                   cudaStream_t stream) {
    static RaisedLimit limit;
    WindowArgs a = args;
    a.stages = plan.stages;
    auto kern = paged_window_decode_small_kernel<Policy>;
    const cudaError_t e = allow_shared_memory(kern, a.device, plan.smem_bytes, &limit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.ctas) * a.num_seqs * a.num_kv_heads);
    cfg.blockDim = dim3(32 * plan.warps);
    cfg.dynamicSmemBytes = static_cast<size_t>(plan.smem_bytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(plan.ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, tmk, tmv);
}

}  // namespace

bool plan_window_small(int num_seqs, int num_kv_heads, int row_blocks, int stage_half_bytes, int num_sms, int max_smem,
                       SmallPlan* plan) {
    const int64_t pairs = static_cast<int64_t>(num_seqs) * num_kv_heads;
    auto bytes = [&](int stages) { return static_cast<int>(warp_bytes(stages, stage_half_bytes)); };
    const int room = max_smem - 8 * 1024;
    // A warp for each block up to eight, as far as shared memory goes; two stages for a warp with several blocks.
    int warps = room / bytes(1);
    if (warps > kMaxWarps) warps = kMaxWarps;
    if (warps > row_blocks) warps = row_blocks;
    if (warps < 1) return false;
    auto stages = [&](int ctas) { return row_blocks > ctas * warps && warps * bytes(2) <= room ? 2 : 1; };
    auto smem = [&](int ctas) { return warps * bytes(stages(ctas)) + 1024; };
    auto per_sm = [&](int ctas) { return 2 * (smem(ctas) + 8 * 1024) <= max_smem ? 2 : 1; };
    // Larger clusters while warps have more than one block and the grid stays within what the SMs hold at once.
    int ctas = 1;
    while (ctas < 8 && row_blocks > ctas * warps) {
        if (2 * ctas * pairs > static_cast<int64_t>(num_sms) * per_sm(2 * ctas)) break;
        ctas *= 2;
    }
    if (pairs * ctas >= (int64_t{1} << 31)) return false;
    plan->warps = warps;
    plan->ctas = ctas;
    plan->stages = stages(ctas);
    plan->smem_bytes = smem(ctas);
    plan->per_sm = per_sm(ctas);
    return true;
}

cudaError_t launch_window_decode_small(const WindowArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                       const SmallPlan& plan, cudaStream_t stream) {
    if (a.kv_dtype == kFP8) {
        const int G = a.num_q_heads / a.num_kv_heads;
        if (a.head_dim != 128) return cudaErrorInvalidValue;
        if (a.dtype == kF16) return launch<MmaFp8Policy<kF16, 128>>(a, tmk, tmv, plan, stream);
        if (a.dtype == kBF16 && G <= 4) return launch<MmaFp8Policy<kBF16, 128, true, 32 * 12>>(a, tmk, tmv, plan, stream);
        if (a.dtype == kBF16) return launch<MmaFp8Policy<kBF16, 128>>(a, tmk, tmv, plan, stream);
        return cudaErrorInvalidValue;
    }
    if (a.dtype == kF16) {
        if (a.head_dim == 64) return launch<MmaPolicy<kF16, 64>>(a, tmk, tmv, plan, stream);
        if (a.head_dim == 128) return launch<MmaPolicy<kF16, 128>>(a, tmk, tmv, plan, stream);
    } else if (a.dtype == kBF16) {
        if (a.head_dim == 64) return launch<MmaPolicy<kBF16, 64>>(a, tmk, tmv, plan, stream);
        if (a.head_dim == 128) return launch<MmaPolicy<kBF16, 128>>(a, tmk, tmv, plan, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pkv
