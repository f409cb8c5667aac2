// Append with the norms of query and key rows and the position rotation on the
// way: each head's row x of a new token becomes, in one pass over the step's rows,
//   z = w x / sqrt(mean(x^2) + eps),   y = the rotation of z by the token's position
// (rope.cu), K rows into the token's slot with V copied beside them, query rows into
// q_out.  The sum of squares, the norm and the rotation are fp32; y is rounded once,
// to the row's type or to an E4M3 code of y / scale.
//
// Work split.  One CTA of 128 threads a token (several, by rows, while there are
// few tokens).  A row belongs to L lanes of a warp, L the power of two from the
// row's items on: an item is V pairs of the rotation (elements i and i + n, or 2i
// and 2i + 1), or 2 V elements behind them, 16 bytes on each side where sizes and
// addresses allow it.  A lane keeps its item in registers from the load to the
// store, so the norm costs log2(L) shuffles and no second look at the row; kRows
// rows are loaded before the first is used.  Weights are read beside the rows, from
// L1 after a CTA's first ones.  Rows of more than 32 items (heads whose sizes leave
// narrow items) take the loop at the end, which reads a row twice.
//
// Bound: HBM.  Every row is read and written once.  16,384 tokens of 32 query and 8 KV
// heads of 128, bf16 (403 MB): 79 us in a graph, 75 % of the rate of a copy, by the ring
// kernel below, whose instructions take 68 % of the issue slots; 105 by the plain one.
// One token: 3.1 us.
#include "rope.cuh"

namespace pkv {

namespace {

// The item `it` of a row: element offsets of its two halves and whether it turns.
struct Item {
    int e0, e1;
    bool turn;
};

template <int V, bool kInter>
__device__ __forceinline__ Item item_of(int it, int nrot, int n) {
    const bool turn = it < nrot;
    const int e0 = turn ? (kInter ? 2 * V * it : V * it) : 2 * n + (it - nrot) * 2 * V;
    return {e0, turn && !kInter ? e0 + n : e0 + V, turn};
}

// V weights of a head from element e on.
template <int DT, int V>
__device__ __forceinline__ void load_weights(const void* w, int64_t e, bool wide, float* f) {
    using T = typename Elem<DT>::T;
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 1.f;
    } else if (wide) {
        const float* p = static_cast<const float*>(w) + e;
        if constexpr (V >= 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(p + i));
                f[i] = x.x, f[i + 1] = x.y, f[i + 2] = x.z, f[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __ldg(p + i);
        }
    } else {
        Raw<V * static_cast<int>(sizeof(T))> r;
        r.load(static_cast<const char*>(w) + e * static_cast<int64_t>(sizeof(T)));
        unpack<DT, V>(r, f);
    }
}

template <int DT, int V, bool kInter, int kRows>
__global__ void __launch_bounds__(kThreads, 5) kv_append_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    static_assert(kThreads >= kMaxRopePairs);
    using T = typename Elem<DT>::T;
    constexpr int kE = static_cast<int>(sizeof(T));
    __shared__ float2 cs[kMaxRopePairs];
    pdl_allow_next();
    pdl_wait();
    const int tid = threadIdx.x;
    const int64_t i = blockIdx.x;  // token
    const int n = a.rot_dim >> 1;
    const int32_t id = a.seq_ids ? a.seq_ids[i] : 0;
    const int32_t slot = a.slot_mapping[i];
    const int32_t pos = tid < n ? a.positions[a.axis[tid] * a.positions_stride + i] : 0;

    const int D = a.head_dim;
    const int nrot = n / V, items = D / (2 * V);
    const int Hq = a.num_q_heads, Hkv = a.num_kv_heads, H = Hq + 2 * Hkv;
    int L = 1;
    while (L < items && L < 32) L <<= 1;
    const int groups = kThreads / L;
    const int my = tid / L, it = tid & (L - 1);
    const int r0 = static_cast<int>(blockIdx.y) * a.rows_per_cta;
    const int r1 = min(H, r0 + a.rows_per_cta);

    auto source = [&](int r) -> const char* {
        if (r < Hq) return static_cast<const char*>(a.q) + (i * a.q_stride + static_cast<int64_t>(r) * D) * kE;
        r -= Hq;
        if (r < Hkv) return static_cast<const char*>(a.k) + (i * a.k_stride + static_cast<int64_t>(r) * D) * kE;
        return static_cast<const char*>(a.v) + (i * a.v_stride + static_cast<int64_t>(r - Hkv) * D) * kE;
    };
    auto weights = [&](int r, int e, float* f) {
        if (r < Hq)
            load_weights<DT, V>(a.q_weight, r * a.q_weight_stride + e, a.wide_weights, f);
        else
            load_weights<DT, V>(a.k_weight, (r - Hq) * a.k_weight_stride + e, a.wide_weights, f);
    };
    const int ce = a.quant ? 1 : kE;  // bytes of a cached element
    const int64_t num_slots = static_cast<int64_t>(a.num_blocks) * a.block_size;
    int blk = 0, off = 0;
    bool keep = false;
    auto target = [&](int r) -> char* {
        if (r < Hq) return static_cast<char*>(a.q_out) + (i * a.q_out_stride + static_cast<int64_t>(r) * D) * kE;
        r -= Hq;
        const bool v = r >= Hkv;
        const int64_t row = (static_cast<int64_t>(blk) * Hkv + (v ? r - Hkv : r)) * a.block_size + off;
        return static_cast<char*>(v ? a.v_cache : a.k_cache) + row * D * ce;
    };
    auto sum_of_squares = [](const float* f) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) s = fmaf(f[j], f[j], s);
        return s;
    };
    const float inv_dim = 1.f / static_cast<float>(D);
    auto factor = [&](float ss) { return rsqrtf(fmaf(ss, inv_dim, a.eps)); };
    // The item's cosines and sines; those of an item that does not turn are 1 and 0.
    auto angles = [&](const Item& x, float2* c) {
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] = x.turn ? cs[x.e0 / (kInter ? 2 : 1) + j] : make_float2(1.f, 0.f);
    };
    // f (an item's 2 V elements) times scale and weights, and turned.
    auto finish = [&](const Item& x, const float2* c, const float* w, float scale, float* f) {
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) f[j] *= w[j];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int ja = kInter ? 2 * j : j, jb = kInter ? 2 * j + 1 : j + V;
            const float xa = f[ja] * scale, xb = f[jb] * scale;
            f[ja] = xa * c[j].x - xb * c[j].y;
            f[jb] = xb * c[j].x + xa * c[j].y;
        }
    };
    auto store = [&](const Item& x, int r, const float* f) {
        char* dst = target(r);
        if (a.quant && r >= Hq) {
            const float scale = r >= Hq + Hkv ? a.v_scale : a.k_scale;
            quantize<V>(f, scale).store(dst + x.e0);
            quantize<V>(f + V, scale).store(dst + x.e1);
        } else {
            pack<DT, V>(f).store(dst + x.e0 * kE);
            pack<DT, V>(f + V).store(dst + x.e1 * kE);
        }
    };

    bool known = false;  // the token's angles and slot (the first time round: every thread of the CTA is here)
    auto know = [&]() -> bool {
        known = true;
        if (tid < n) cs[tid] = rotor(static_cast<uint64_t>(static_cast<int64_t>(pos)) * a.phase[tid], a.amplitude);
        __syncthreads();
        keep = slot >= 0 && slot < num_slots;
        if (id >= 0 && slot >= num_slots && tid == 0 && blockIdx.y == 0) raise_flag(a.status, kFlagBadSlot);
        blk = keep ? slot / a.block_size : 0;
        off = slot - blk * a.block_size;
        return id >= 0;
    };

    if (items <= 32) {
        const Item x = item_of<V, kInter>(it, nrot, n);
        const bool active = it < items;
        float2 c[V];
        for (int rb = r0; rb < r1; rb += groups * kRows) {
            Raw<V * kE> x0[kRows], x1[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int r = rb + u * groups + my;
                if (active && r < r1) {
                    const char* src = source(r);
                    x0[u].load(src + x.e0 * kE);
                    x1[u].load(src + x.e1 * kE);
                }
            }
            if (!known) {
                if (!know()) return;  // padding
                if (active) angles(x, c);
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int r = rb + u * groups + my;
                const bool mine = active && r < r1;
                float f[2 * V];
                float ss = 0.f;
                if (mine) {
                    unpack<DT, V>(x0[u], f);
                    unpack<DT, V>(x1[u], f + V);
                    ss = sum_of_squares(f);
                }
                for (int o = L >> 1; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (!mine || (r >= Hq && !keep)) continue;
                if (r >= Hq + Hkv) {  // a V row
                    if (a.quant) {
                        store(x, r, f);
                    } else {  // bit for bit
                        char* dst = target(r);
                        x0[u].store(dst + x.e0 * kE);
                        x1[u].store(dst + x.e1 * kE);
                    }
                    continue;
                }
                float w[2 * V];
                weights(r, x.e0, w);
                weights(r, x.e1, w + V);
                finish(x, c, w, factor(ss), f);
                store(x, r, f);
            }
        }
        return;
    }
    // More items than lanes: a warp a row, which is read again for its second use.
    if (!know()) return;
    for (int r = r0 + my; r < r1; r += groups) {
        const char* src = source(r);
        float ss = 0.f;
        if (r < Hq + Hkv) {
            for (int k = it; k < items; k += 32) {
                const Item x = item_of<V, kInter>(k, nrot, n);
                Raw<V * kE> x0, x1;
                float f[2 * V];
                x0.load(src + x.e0 * kE);
                x1.load(src + x.e1 * kE);
                unpack<DT, V>(x0, f);
                unpack<DT, V>(x1, f + V);
                ss += sum_of_squares(f);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        if (r >= Hq && !keep) continue;
        const float scale = factor(ss);
        for (int k = it; k < items; k += 32) {
            const Item x = item_of<V, kInter>(k, nrot, n);
            Raw<V * kE> x0, x1;
            float f[2 * V];
            x0.load(src + x.e0 * kE);
            x1.load(src + x.e1 * kE);
            unpack<DT, V>(x0, f);
            unpack<DT, V>(x1, f + V);
            if (r < Hq + Hkv) {
                float w[2 * V];
                weights(r, x.e0, w);
                weights(r, x.e1, w + V);
                float2 c[V];
                angles(x, c);
                finish(x, c, w, scale, f);
            } else if (!a.quant) {
                char* dst = target(r);
                x0.store(dst + x.e0 * kE);
                x1.store(dst + x.e1 * kE);
                continue;
            }
            store(x, r, f);
        }
    }
}

constexpr int kRing = 2;  // tokens in shared memory

// The same for many tokens whose rows are whole 16-byte chunks: persistent CTAs that
// bring the rows of a token (three contiguous pieces: q, k, v) into shared memory by
// bulk copies while they work on the token before, so that loads never pause and no
// register waits for one.  Two tokens, six CTAs an SM: deeper rings and other counts
// took 81 to 103 us for 16,384 tokens, two elements an instruction 81.
template <int DT, bool kInter>
__global__ void __launch_bounds__(kThreads, 6) kv_append_norm_rope_ring_kernel(const __grid_constant__ NormRopeArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int kE = static_cast<int>(sizeof(T)), V = 16 / kE;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t full[kRing];
    __shared__ int abort_flag;
    __shared__ float2 cs[2][kMaxRopePairs];
    volatile int* abort = &abort_flag;
    pdl_allow_next();
    const int tid = threadIdx.x;
    const int n = a.rot_dim >> 1;
    const int D = a.head_dim, Hq = a.num_q_heads, Hkv = a.num_kv_heads, H = Hq + 2 * Hkv;
    const uint32_t row = static_cast<uint32_t>(D) * kE;
    const uint32_t bytes = static_cast<uint32_t>(H) * row;
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
        *abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    const uint64_t policy = policy_evict_first();
    auto fetch = [&](int64_t i, uint32_t stage) {  // thread 0
        uint8_t* dst = ring + stage * bytes;
        mbar_arrive_expect_tx(&full[stage], bytes);
        if (Hq) bulk_load(dst, static_cast<const char*>(a.q) + i * a.q_stride * kE, Hq * row, &full[stage], policy);
        bulk_load(dst + Hq * row, static_cast<const char*>(a.k) + i * a.k_stride * kE, Hkv * row, &full[stage], policy);
        bulk_load(dst + (Hq + Hkv) * row, static_cast<const char*>(a.v) + i * a.v_stride * kE, Hkv * row, &full[stage], policy);
    };
    const int64_t step = gridDim.x;
    if (tid == 0)
        for (int k = 0; k < kRing; ++k)
            if (blockIdx.x + k * step < a.n_tokens) fetch(blockIdx.x + k * step, k);

    const int nrot = n / V, items = D / (2 * V);
    int L = 1;
    while (L < items) L <<= 1;
    const int groups = kThreads / L;
    const int my = tid / L, it = tid & (L - 1);
    const bool active = it < items;
    const Item x = item_of<V, kInter>(it, nrot, n);
    const float inv_dim = 1.f / static_cast<float>(D);
    const int ce = a.quant ? 1 : kE;
    const int64_t num_slots = static_cast<int64_t>(a.num_blocks) * a.block_size;
    const int32_t* my_positions = a.positions + (tid < n ? a.axis[tid] * a.positions_stride : 0);
    const uint64_t my_phase = tid < n ? a.phase[tid] : 0;
    // What the next token is, asked for a token ahead.
    int32_t id = 0, slot = 0, pos = 0;
    auto ask = [&](int64_t i) {
        if (i >= a.n_tokens) return;
        id = a.seq_ids ? a.seq_ids[i] : 0;
        slot = a.slot_mapping[i];
        if (tid < n) pos = my_positions[i];
    };
    auto turn = [&](int k) {
        if (tid < n) cs[k][tid] = rotor(static_cast<uint64_t>(static_cast<int64_t>(pos)) * my_phase, a.amplitude);
    };
    ask(blockIdx.x);
    turn(0);
    __syncthreads();
    uint32_t stage = 0, round = 0;
    int k = 0;
    for (int64_t i = blockIdx.x; i < a.n_tokens; i += step) {
        const int32_t now_id = id, now_slot = slot;
        ask(i + step);
        float2 c[V];
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] = active && x.turn ? cs[k][x.e0 / (kInter ? 2 : 1) + j] : make_float2(1.f, 0.f);
        const bool keep = now_slot >= 0 && now_slot < num_slots;
        if (now_id >= 0 && now_slot >= num_slots && tid == 0) raise_flag(a.status, kFlagBadSlot);
        const int blk = keep ? now_slot / a.block_size : 0, off = now_slot - blk * a.block_size;
        if (!mbar_wait_bounded(&full[stage], round & 1u, abort, a.status)) break;
        const uint8_t* src = ring + stage * bytes;
        if (now_id >= 0) {
            for (int rb = 0; rb < H; rb += groups) {
                const int r = rb + my;
                const bool mine = active && r < H;
                Raw<16> x0, x1;
                float f[2 * V];
                float ss = 0.f;
                if (mine) {
                    x0.load(reinterpret_cast<const char*>(src) + r * row + x.e0 * kE);
                    x1.load(reinterpret_cast<const char*>(src) + r * row + x.e1 * kE);
                    unpack<DT, V>(x0, f);
                    unpack<DT, V>(x1, f + V);
#pragma unroll
                    for (int j = 0; j < 2 * V; ++j) ss = fmaf(f[j], f[j], ss);
                }
                for (int o = L >> 1; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (!mine || (r >= Hq && !keep)) continue;
                const bool copy = r >= Hq + Hkv;
                char* dst;
                if (r < Hq) {
                    dst = static_cast<char*>(a.q_out) + (i * a.q_out_stride + static_cast<int64_t>(r) * D) * kE;
                } else {
                    const int h = r - Hq - (copy ? Hkv : 0);
                    const int64_t at = (static_cast<int64_t>(blk) * Hkv + h) * a.block_size + off;
                    dst = static_cast<char*>(copy ? a.v_cache : a.k_cache) + at * D * ce;
                }
                if (!copy) {
                    float w[2 * V];
                    const void* wp = r < Hq ? a.q_weight : a.k_weight;
                    const int64_t w0 = r < Hq ? r * a.q_weight_stride : (r - Hq) * a.k_weight_stride;
                    load_weights<DT, V>(wp, w0 + x.e0, a.wide_weights, w);
                    load_weights<DT, V>(wp, w0 + x.e1, a.wide_weights, w + V);
                    const float scale = rsqrtf(fmaf(ss, inv_dim, a.eps));
#pragma unroll
                    for (int j = 0; j < 2 * V; ++j) f[j] *= w[j];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int ja = kInter ? 2 * j : j, jb = kInter ? 2 * j + 1 : j + V;
                        const float xa = f[ja] * scale, xb = f[jb] * scale;
                        f[ja] = xa * c[j].x - xb * c[j].y;
                        f[jb] = xb * c[j].x + xa * c[j].y;
                    }
                } else if (!a.quant) {  // bit for bit
                    x0.store(dst + x.e0 * kE);
                    x1.store(dst + x.e1 * kE);
                    continue;
                }
                if (a.quant && r >= Hq) {
                    const float scale = copy ? a.v_scale : a.k_scale;
                    quantize<V>(f, scale).store(dst + x.e0);
                    quantize<V>(f + V, scale).store(dst + x.e1);
                } else {
                    pack<DT, V>(f).store(dst + x.e0 * kE);
                    pack<DT, V>(f + V).store(dst + x.e1 * kE);
                }
            }
        }
        if (i + step < a.n_tokens) turn(k ^ 1);
        __syncthreads();  // the stage and cs[k] are read, cs[k ^ 1] is there
        if (tid == 0 && i + kRing * step < a.n_tokens) fetch(i + kRing * step, stage);
        k ^= 1;
        if (++stage == kRing) {
            stage = 0;
            ++round;
        }
    }
    // (Every copy that was issued has been waited for, unless a wait gave up.)
    if (*abort && tid == 0)
        for (int q = 0; q < kRing; ++q) {
            const uint64_t t0 = global_timer_ns();
            const uint32_t parity = (round + (static_cast<uint32_t>(q) < stage ? 1u : 0u)) & 1u;
            while (!mbar_try_wait(&full[q], parity) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
}

// CTAs of the ring kernel that an SM holds, tokens of `bytes` bytes.
int ring_ctas(int bytes) {
    const int fit = (220 * 1024) / (kRing * bytes + 4096);
    return fit < 6 ? fit : 6;
}

template <int DT>
cudaError_t launch_ring(const NormRopeArgs& a, int bytes, int num_sms, cudaStream_t stream) {
    static RaisedLimit limits[2];
    auto kern = a.interleaved ? kv_append_norm_rope_ring_kernel<DT, true> : kv_append_norm_rope_ring_kernel<DT, false>;
    const int smem = kRing * bytes;
    const cudaError_t e = allow_shared_memory(kern, a.device, smem, &limits[a.interleaved ? 1 : 0]);
    if (e != cudaSuccess) return e;
    const int64_t ctas = static_cast<int64_t>(num_sms) * ring_ctas(bytes);
    return launch_kernel(kern, dim3(static_cast<unsigned>(ctas < a.n_tokens ? ctas : a.n_tokens)), dim3(kThreads),
                         static_cast<size_t>(smem), stream, a.pdl != 0, a);
}

template <int DT, int V, int kRows>
cudaError_t launch_v(const NormRopeArgs& a, dim3 grid, cudaStream_t stream) {
    if (a.interleaved)
        return launch_kernel(kv_append_norm_rope_kernel<DT, V, true, kRows>, grid, dim3(kThreads), 0, stream, a.pdl != 0, a);
    return launch_kernel(kv_append_norm_rope_kernel<DT, V, false, kRows>, grid, dim3(kThreads), 0, stream, a.pdl != 0, a);
}

template <int DT>
cudaError_t launch_dt(NormRopeArgs a, int align, int weight_align, int num_sms, cudaStream_t stream) {
    constexpr int kE = static_cast<int>(sizeof(typename Elem<DT>::T));
    auto weights_fit = [&](int v) {
        const int need = a.wide_weights ? (v >= 4 ? 16 : 4) : v * kE;
        return (!a.q_weight && !a.k_weight) || weight_align >= need;
    };
    int v = 16 / kE;
    while (v > 1 && ((a.rot_dim / 2) % v || (a.head_dim - a.rot_dim) % (2 * v) || a.head_dim % v || align < v * kE ||
                     !weights_fit(v)))
        v >>= 1;
    const int items = a.head_dim / (2 * v);
    // Many tokens of whole 16-byte items: the ring, while three of its CTAs fit an SM.  Its time goes in rounds of one
    // token a CTA, so with few CTAs an SM, or f32 rows, it is ahead in the first round where that is nearly full, and
    // then only from many rounds on.  Ring / plain kernel, us in graphs, heads of 128 and 8 KV heads:
    //   bf16, 32 query heads (six CTAs an SM): 304 tokens 4.4 / 5.9, 608 6.5 / 6.1, 912 6.5 / 9.9, 1,216 10.7 / 10.6,
    //     4,096 24.9 / 29.0, 16,384 78.9 / 103; f16 into E4M3: 1,023 9.9 / 11.8, 16,384 87.5 / 118;
    //   64 (five): 304 7.7 / 6.3, 456 8.0 / 8.9, 1,023 15.4 / 14.2, 4,096 38 / 48; 80 (four): 1,023 16.5 / 15.7, 4,096 47 / 54;
    //   112 (three): 456 9.5 / 10.5, 608 17.1 / 14.0, 1,023 24.5 / 20.8, 2,048 38.6 / 37.6, 4,096 65 / 73; 128 (two): 456
    //     15.7 / 11.1, 16,384 382 / 303;
    //   f32, 32 (four): 304 5.4 / 4.9, 608 6.9 / 8.4, 1,023 14.0 / 12.4, 2,048 24.7 / 22.0, 4,096 40 / 43, 16,384 138 / 165.
    const int64_t bytes = static_cast<int64_t>(a.num_q_heads + 2 * a.num_kv_heads) * a.head_dim * kE;
    if (v == 16 / kE && items <= 32 && kRing * bytes <= 69 * 1024) {
        const int per_sm = ring_ctas(static_cast<int>(bytes));
        const int each = (a.n_tokens - 1) / num_sms + 1;  // tokens an SM
        const bool first_round = each <= per_sm && each >= (kE == 4 ? 4 : 3);
        const int from = kE == 4 ? 24 : per_sm >= 6 ? 2 : per_sm >= 4 ? 3 : 16;
        if (first_round || a.n_tokens >= from * num_sms)
            return launch_ring<DT>(a, static_cast<int>(bytes), num_sms, stream);
    }
    int L = 1;
    while (L < items && L < 32) L <<= 1;
    const int groups = kThreads / L;
    const int H = a.num_q_heads + 2 * a.num_kv_heads;
    // As in rope.cu: the rows that the threads load in one round, two or three a
    // thread, one while that leaves no more CTAs than two for each SM.
    const int passes = (H + groups - 1) / groups;
    int per = (passes + 2) / 3 < (passes + 1) / 2 ? 3 : 2;
    while (per > 1 && static_cast<int64_t>(a.n_tokens) * ((passes + per - 2) / (per - 1)) <= 2 * num_sms) --per;
    while ((passes + per - 1) / per > 65535) per *= 2;  // the grid's limit in y
    a.rows_per_cta = per * groups;
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

cudaError_t launch_append_norm_rope(const NormRopeArgs& a, int align, int weight_align, int num_sms,
                                    cudaStream_t stream) {
    switch (a.src_dtype) {
        case kF32: return launch_dt<kF32>(a, align, weight_align, num_sms, stream);
        case kF16: return launch_dt<kF16>(a, align, weight_align, num_sms, stream);
        case kBF16: return launch_dt<kBF16>(a, align, weight_align, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
