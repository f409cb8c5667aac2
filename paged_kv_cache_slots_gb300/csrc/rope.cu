// Append with the position rotation applied on the way: each new token's K
// rows are rotated and written to the token's slot, its V rows copied beside
// them, and its query rows rotated into q_out, in one pass over the step's
// rows (the slot rule is that of append.cu; "vLLM Architecture and
// Installation", Example 3).
//
// The rotation.  Pair i < n of a head (n = rot_dim / 2; elements (i, i + n),
// or (2i, 2i + 1) when interleaved) turns by t = p * f_i, p the token's
// position on the pair's axis:
//   y_a = A (x_a cos t - x_b sin t),  y_b = A (x_b cos t + x_a sin t);
// elements from rot_dim on are copied.  Computed in fp32 and rounded once, to
// the row's type or to an E4M3 code of y / scale.
//
// The angle.  p * f_i in fp32 is off by up to p * f_i * 2^-24 radians, which
// at far positions is larger than the angles between neighbours.  The host
// turns f_i into a fraction of a turn in 64-bit fixed point
// (F_i = f_i / 2 pi * 2^64 mod 2^64), so p * F_i mod 2^64 is the angle's
// fraction of a turn to p * 2^-64: one integer multiplication, with no
// reduction and no table of positions to read.  The nearest quarter turn is
// taken off in integers, and sincospif sees at most an eighth of a turn, where
// the conversion to fp32 is off by at most 2^-28 of a turn.
//
// Work split.  One CTA of 128 threads a token (several, by rows, when there
// are too few tokens to fill the GPU).  The first n threads make the token's
// cosines and sines in shared memory while the first rows' loads are in
// flight.  A thread keeps one item of a row -- V pairs, 2 V elements -- and
// walks the token's rows (Hq query, Hkv K, Hkv V) with it, so its cosines and
// sines stay in registers; kRows rows are loaded before the first is used.
// V pairs are 16 bytes on each side where sizes and addresses allow it.
//
// Bound: HBM.  Every row is read and written once: 16,384 tokens of 32 query
// and 8 KV heads of 128 bf16 elements move 403 MB in 68 us, 5.9 TB/s (88 % of
// the measured copy rate; 112 us when the slot and the padding flag were waited
// for before the rows were asked for).  Small calls are bound by their launch and
// two rounds of loads (2.3 us for one token).
//
// Registers are bounded for seven CTAs an SM (72 each) in every variant.  In a
// graph, with 6 / 7 / 8 CTAs: the chunk above 72.1 / 67.7 / 71.4 us, 1,023 tokens
// into E4M3 6.6 / 5.1 / 5.5, 4,099 tokens of 16 and 2 heads on three axes 13.9 /
// 13.7 / 13.3, f32 heads of 80 10.2 / 9.6 / 9.4.  Seven costs the variants of eight
// 16-bit elements and three rows 24 bytes of spills.
#include "device_utils.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;  // kMaxRopePairs: a thread makes one cosine and sine at most

// V elements of T as raw words.
template <int kBytes>
struct Raw {
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const char* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (kBytes == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint8_t*>(p);
        }
    }
    __device__ __forceinline__ void store(char* p) const {
        if constexpr (kBytes == 16)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else if constexpr (kBytes == 2)
            *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
        else
            *reinterpret_cast<uint8_t*>(p) = static_cast<uint8_t>(w[0]);
    }
};

template <int DT, int V>
__device__ __forceinline__ void unpack(const Raw<V * static_cast<int>(sizeof(typename Elem<DT>::T))>& r, float* f) {
    using T = typename Elem<DT>::T;
    const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = Elem<DT>::to_float(e[i]);
}

template <int DT, int V>
__device__ __forceinline__ Raw<V * static_cast<int>(sizeof(typename Elem<DT>::T))> pack(const float* f) {
    using T = typename Elem<DT>::T;
    Raw<V * static_cast<int>(sizeof(T))> r;
    T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = Elem<DT>::from_float(f[i]);
    return r;
}

// E4M3 codes of V values / scale (as kv_append_fp8).
template <int V>
__device__ __forceinline__ Raw<V> quantize(const float* f, float scale) {
    Raw<V> r;
    if constexpr (V == 1) {
        r.w[0] = e4m3x2_from_floats(__fdiv_rn(f[0], scale), 0.f) & 0xFFu;
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const uint32_t c = e4m3x2_from_floats(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale));
            if (i & 1)
                r.w[i / 2] |= c << 16;
            else
                r.w[i / 2] = c;
        }
    }
    return r;
}

// Cosine and sine of `turn` (a fraction of a turn times 2^64, as a signed
// number), times `amplitude`.
__device__ __forceinline__ float2 rotor(uint64_t turn, float amplitude) {
    const int32_t t = static_cast<int32_t>((turn + 0x80000000ull) >> 32);  // to 2^-32 of a turn, nearest
    const uint32_t quarter = (static_cast<uint32_t>(t) + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(t) - (quarter << 30));  // at most 2^29
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    const float cq = (quarter & 1u) ? s : c, sq = (quarter & 1u) ? c : s;
    // Quarter turns 1 and 2 flip the cosine's sign, 2 and 3 the sine's.
    const float cs = (quarter == 1u || quarter == 2u) ? -cq : cq;
    const float sn = quarter >= 2u ? -sq : sq;
    return make_float2(cs * amplitude, sn * amplitude);
}

// kRows: rows a thread loads before it uses the first.
template <int DT, int V, bool kInter, int kRows>
__global__ void __launch_bounds__(kThreads, 7) kv_append_rope_kernel(const __grid_constant__ RopeArgs a) {
    static_assert(kThreads >= kMaxRopePairs);
    using T = typename Elem<DT>::T;
    constexpr int kE = static_cast<int>(sizeof(T));
    __shared__ float2 cs[kMaxRopePairs];
    pdl_allow_next();
    pdl_wait();
    const int tid = threadIdx.x;
    const int64_t i = blockIdx.x;  // token
    const int n = a.rot_dim >> 1;
    // What the token is, its positions and its first rows are asked for at
    // once; nothing waits for an answer before the loads are on their way.
    const int32_t id = a.seq_ids ? a.seq_ids[i] : 0;
    const int32_t slot = a.slot_mapping[i];
    const int32_t pos = tid < n ? a.positions[a.axis[tid] * a.positions_stride + i] : 0;

    const int nrot = n / V;                             // items of V pairs
    const int items = nrot + (a.head_dim - 2 * n) / V;  // and items of V copied elements
    const int Hq = a.num_q_heads, Hkv = a.num_kv_heads, H = Hq + 2 * Hkv;
    const int slots = items < kThreads ? kThreads / items : 1;  // rows taken side by side
    const int my = items < kThreads ? tid / items : 0;
    const int r0 = static_cast<int>(blockIdx.y) * a.rows_per_cta;
    const int r1 = min(H, r0 + a.rows_per_cta);

    auto source = [&](int r) -> const char* {
        if (r < Hq) return static_cast<const char*>(a.q) + (i * a.q_stride + static_cast<int64_t>(r) * a.head_dim) * kE;
        r -= Hq;
        if (r < Hkv) return static_cast<const char*>(a.k) + (i * a.k_stride + static_cast<int64_t>(r) * a.head_dim) * kE;
        return static_cast<const char*>(a.v) + (i * a.v_stride + static_cast<int64_t>(r - Hkv) * a.head_dim) * kE;
    };
    const int ce = a.quant ? 1 : kE;  // bytes of a cached element
    const int64_t num_slots = static_cast<int64_t>(a.num_blocks) * a.block_size;
    int blk = 0, off = 0;
    bool keep = false;
    auto target = [&](int r) -> char* {
        if (r < Hq)
            return static_cast<char*>(a.q_out) + (i * a.q_out_stride + static_cast<int64_t>(r) * a.head_dim) * kE;
        r -= Hq;
        const bool v = r >= Hkv;
        const int64_t row = (static_cast<int64_t>(blk) * Hkv + (v ? r - Hkv : r)) * a.block_size + off;
        return static_cast<char*>(v ? a.v_cache : a.k_cache) + row * a.head_dim * ce;
    };

    bool angles = false;
    for (int it0 = 0; it0 < items; it0 += kThreads) {
        const int it = items < kThreads ? tid - my * items : it0 + tid;
        const bool active = my < slots && it < items;
        const bool turn = it < nrot;  // else a copied item
        const int e0 = turn ? (kInter ? 2 * V * it : V * it) : 2 * n + (it - nrot) * V;
        const int e1 = kInter ? e0 + V : e0 + n;  // second half of a turned item
        float2 w[V];
        for (int rb = r0; rb < r1; rb += slots * kRows) {
            Raw<V * kE> x0[kRows], x1[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int r = rb + u * slots + my;
                if (active && r < r1) {
                    const char* src = source(r);
                    x0[u].load(src + e0 * kE);
                    if (turn) x1[u].load(src + e1 * kE);
                }
            }
            if (!angles) {  // the first time round: every thread of the CTA is here
                angles = true;
                if (tid < n) cs[tid] = rotor(static_cast<uint64_t>(static_cast<int64_t>(pos)) * a.phase[tid], a.amplitude);
                __syncthreads();
                if (id < 0) return;  // padding
                keep = slot >= 0 && slot < num_slots;
                if (slot >= num_slots && tid == 0 && blockIdx.y == 0) raise_flag(a.status, kFlagBadSlot);
                blk = keep ? slot / a.block_size : 0;
                off = slot - blk * a.block_size;
            }
            if (rb == r0 && active && turn) {
#pragma unroll
                for (int j = 0; j < V; ++j) w[j] = cs[V * it + j];
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int r = rb + u * slots + my;
                if (!active || r >= r1 || (r >= Hq && !keep)) continue;
                char* dst = target(r);
                const bool copy = r >= Hq + Hkv;  // a V row
                const bool codes = a.quant && r >= Hq;
                if (!codes && (copy || !turn)) {  // bit for bit
                    x0[u].store(dst + e0 * kE);
                    if (turn) x1[u].store(dst + e1 * kE);
                    continue;
                }
                float f[2 * V];
                unpack<DT, V>(x0[u], f);
                if (turn) {
                    unpack<DT, V>(x1[u], f + V);
                    if (!copy) {
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const int ja = kInter ? 2 * j : j, jb = kInter ? 2 * j + 1 : j + V;
                            const float xa = f[ja], xb = f[jb];
                            f[ja] = xa * w[j].x - xb * w[j].y;
                            f[jb] = xb * w[j].x + xa * w[j].y;
                        }
                    }
                }
                if (codes) {
                    const float scale = copy ? a.v_scale : a.k_scale;
                    quantize<V>(f, scale).store(dst + e0);
                    if (turn) quantize<V>(f + V, scale).store(dst + e1);
                } else {
                    pack<DT, V>(f).store(dst + e0 * kE);
                    pack<DT, V>(f + V).store(dst + e1 * kE);
                }
            }
        }
    }
}

template <int DT, int V, int kRows>
cudaError_t launch_v(const RopeArgs& a, dim3 grid, cudaStream_t stream) {
    if (a.interleaved)
        return launch_kernel(kv_append_rope_kernel<DT, V, true, kRows>, grid, dim3(kThreads), 0, stream, a.pdl != 0, a);
    return launch_kernel(kv_append_rope_kernel<DT, V, false, kRows>, grid, dim3(kThreads), 0, stream, a.pdl != 0, a);
}

// Pairs an item holds: 16 bytes a side, or as many as the sizes and the
// addresses (`align`: the power of two that divides every row's address)
// leave whole.
template <int DT>
cudaError_t launch_dt(RopeArgs a, int align, int num_sms, cudaStream_t stream) {
    constexpr int kE = static_cast<int>(sizeof(typename Elem<DT>::T));
    int v = 16 / kE;
    while (v > 1 && ((a.rot_dim / 2) % v || a.head_dim % v || align < v * kE)) v >>= 1;
    const int items = (a.head_dim - a.rot_dim / 2) / v;
    const int slots = items < kThreads ? kThreads / items : 1;
    const int H = a.num_q_heads + 2 * a.num_kv_heads;
    // A CTA takes the rows of one token that its threads load in one round, two
    // or three rows a thread (three where that takes fewer CTAs), one while
    // that leaves no more CTAs than two for each SM: with few tokens a call is
    // bound by its latency.
    const int passes = (H + slots - 1) / slots;
    int per = (passes + 2) / 3 < (passes + 1) / 2 ? 3 : 2;
    while (per > 1 && static_cast<int64_t>(a.n_tokens) * ((passes + per - 2) / (per - 1)) <= 2 * num_sms) --per;
    while ((passes + per - 1) / per > 65535) per *= 2;  // the grid's limit in y
    a.rows_per_cta = per * slots;
    const dim3 grid(static_cast<unsigned>(a.n_tokens), static_cast<unsigned>((passes + per - 1) / per));
    const bool three = per >= 3;
    switch (v) {
        case 8:
            if constexpr (kE == 2) return three ? launch_v<DT, 8, 3>(a, grid, stream) : launch_v<DT, 8, 2>(a, grid, stream);
            return cudaErrorInvalidValue;
        case 4: return three ? launch_v<DT, 4, 3>(a, grid, stream) : launch_v<DT, 4, 2>(a, grid, stream);
        case 2: return three ? launch_v<DT, 2, 3>(a, grid, stream) : launch_v<DT, 2, 2>(a, grid, stream);
        default: return three ? launch_v<DT, 1, 3>(a, grid, stream) : launch_v<DT, 1, 2>(a, grid, stream);
    }
}

}  // namespace

cudaError_t launch_append_rope(const RopeArgs& a, int align, int num_sms, cudaStream_t stream) {
    switch (a.src_dtype) {
        case kF32: return launch_dt<kF32>(a, align, num_sms, stream);
        case kF16: return launch_dt<kF16>(a, align, num_sms, stream);
        case kBF16: return launch_dt<kBF16>(a, align, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
