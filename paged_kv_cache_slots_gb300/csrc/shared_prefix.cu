// The merge of the shared-prefix attention's parts and the choice of its
// kernels (see shared_prefix_kernel.cuh).
#include "prefix_units.cuh"
#include "shared_prefix.cuh"

namespace pkv {

namespace {

// One warp a (sequence, query head): the prefix's parts, then the parts that
// the tails left.  Lane l holds (max, sum) and the row of part l of 32; every
// lane sums D / 32 output elements, four parts' loads at a time, the first four
// asked for together with the (max, sum) pairs.  Bound by the latency of its
// two rounds of loads: few registers, so that many warps wait at once.
template <int D>
__global__ void __launch_bounds__(256, 4) shared_prefix_merge_kernel(const SharedPrefixArgs a, const TailArgs d) {
    constexpr int VD = D / 32;
    pdl_allow_next();
    pdl_wait();
    const int row = static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= a.num_seqs * a.num_q_heads) return;
    const int s = row / a.num_q_heads;
    const int hq = row - s * a.num_q_heads;
    const int G = a.num_q_heads / a.num_kv_heads;
    const int h = hq / G, g = hq - h * G;
    const int Hc = d.heads_per_stage;
    const int hc = h / Hc, hw = h - hc * Hc;
    const int pair = s * (d.num_kv_heads / Hc) + hc;
    const int4 pp = a.parts[s * a.num_kv_heads + h];
    const int4 tp = d.tail_parts[pair];
    const int n = pp.z + tp.y;
    float M = -INFINITY, L = 0.f, acc[VD];
#pragma unroll
    for (int i = 0; i < VD; ++i) acc[i] = 0.f;
    for (int base = 0; base < n; base += 32) {
        // This lane's part: its row among all partial rows (the tails' follow the prefix's).
        const int p = base + lane;
        int r = -1;
        if (p < pp.z) {
            r = pp.x + p * pp.y + g;
            if (r >= a.max_rows) r = -1;
        } else if (p < n) {
            const int k = p - pp.z;
            const int c = tp.w == 0 ? tp.x + k : cta_of_tile(tp.z + k, tp.w, tp.x);
            r = a.max_rows + ((c + pair) * Hc + hw) * G + g;
        }
        const int cnt = min(32, n - base);
        float v[4][VD];
        auto fetch = [&](int k0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int rk = __shfl_sync(0xffffffffu, r, (k0 + k) & 31);
                const bool get = k0 + k < cnt && rk >= 0;
                const float* src = a.part_o + static_cast<int64_t>(get ? rk : 0) * D;
                if constexpr (VD == 4) {
                    const float4 t = get ? __ldcg(reinterpret_cast<const float4*>(src) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[k][0] = t.x, v[k][1] = t.y, v[k][2] = t.z, v[k][3] = t.w;
                } else {
                    const float2 t = get ? __ldcg(reinterpret_cast<const float2*>(src) + lane) : make_float2(0.f, 0.f);
                    v[k][0] = t.x, v[k][1] = t.y;
                }
            }
        };
        const float2 ml = r >= 0 ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + r) : make_float2(-INFINITY, 0.f);
        fetch(0);
        float mx = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float Mn = fmaxf(M, mx);
        const float w = r >= 0 ? fast_exp2(ml.x - Mn) : 0.f;
        const float al = base == 0 ? 0.f : fast_exp2(M - Mn);
        float ls = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        L = L * al + ls;
        M = Mn;
#pragma unroll
        for (int i = 0; i < VD; ++i) acc[i] *= al;
#pragma unroll 1
        for (int k0 = 0; k0 < cnt; k0 += 4) {
            if (k0 > 0) fetch(k0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                if (k0 + k < cnt) {
#pragma unroll
                    for (int i = 0; i < VD; ++i) acc[i] = fmaf(wk, v[k][i], acc[i]);
                }
            }
        }
    }
    const float inv = n > 0 ? 1.f / L : 0.f;  // a sequence without tokens: zeros
    const int64_t o0 = static_cast<int64_t>(row) * D + lane * VD;
#pragma unroll
    for (int i = 0; i < VD; ++i) acc[i] = n > 0 ? acc[i] * inv : 0.f;
    if (a.out_dtype == kF32) {
        float* o = static_cast<float*>(a.out) + o0;
        if constexpr (VD == 4)
            *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else
            *reinterpret_cast<float2*>(o) = make_float2(acc[0], acc[1]);
        return;
    }
    uint32_t w[VD / 2];
#pragma unroll
    for (int i = 0; i < VD / 2; ++i) {
        if (a.out_dtype == kF16) {
            const __half2 h = __floats2half2_rn(acc[2 * i], acc[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    char* o = static_cast<char*>(a.out) + o0 * 2;
    if constexpr (VD == 4)
        *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t*>(o) = w[0];
}

template <int D>
cudaError_t launch_merge_t(const SharedPrefixArgs& a, const TailArgs& tails, cudaStream_t stream) {
    static RaisedLimit carveout;
    auto kern = shared_prefix_merge_kernel<D>;
    const cudaError_t e = prefer_shared_memory(kern, tails.device, &carveout);
    if (e != cudaSuccess) return e;
    const int64_t warps = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
    return launch_kernel(kern, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0, stream, true, a, tails);
}

}  // namespace

cudaError_t launch_shared_prefix(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmk,
                                 const CUtensorMap& tmv, cudaStream_t stream) {
    cudaError_t e = d.kv_dtype == kFP8    ? launch_attend_fp8(a, d, tmk, tmv, stream)
                    : d.dtype == kBF16 ? launch_attend_bf16(a, d, tmk, tmv, stream)
                                       : launch_attend_f16(a, d, tmk, tmv, stream);
    if (e != cudaSuccess) return e;
    if (a.head_dim == 64) return launch_merge_t<64>(a, d, stream);
    return launch_merge_t<128>(a, d, stream);
}

}  // namespace pkv
