// Chunks of new tokens under a sliding window on the fifth-generation tensor cores
// (tcgen05): f16 and bf16 caches (see paged_window_prefill_attention).
//
// For a row (new token at position p, query head g) over the keys j in sight,
// j <= p and (j > p - window or j < sinks):
//   s_j = scale q . k_j,  m = max s_j,  out = sum 2^(s_j - m) v_j / sum 2^(s_j - m)
// in base 2, with one pass over the keys: the running reference m only moves when a
// row's maximum grows by more than 2^8 (the weights stay <= 256), and O and the sum
// are rescaled then.
//
// Work split.  An item is 256 / G new tokens of one sequence with the G query heads
// of one KV head: 256 rows, two tiles of 128, so that a K and V tile read from L2
// serves 256 rows (at 128 rows a CTA the tensor cores would ask L2 for twice as much
// as it gives).  A persistent CTA for each SM walks its items; the keys of an item
// are a list of boxes of 16 or 32 rows of a cached block (those of the first tokens,
// then those of the window), taken 128 keys at a time:
//   warp 8       producer: Q, K and V by TMA into a Q buffer and a ring of stages
//                (a stage is the K or the V of 128 keys), ahead into the next item;
//   warp 9       (one lane) issues the MMAs.  S = Q . K^T of one row tile (M 128,
//                N 128) while the other's softmax runs, then O += P . V with P read
//                from tensor memory over the S it came from;
//   warps 0-3, 4-7  softmax of the two row tiles, a thread a row: load S, mask (the
//                tiles at the edges of the window alone), maximum, weights, P; at the
//                end of an item O / l.
// The MMAs run in the order of their issue, so that S of the next keys being there
// says that P . V of these is done: the rescaling of O needs no wait of its own.
//
// Roundings.  S, O, the maxima and sums are fp32.  With a 16-bit output a weight
// meets V rounded to q's type (half a step: as much as the output's own rounding),
// with an fp32 output in two parts, which hold it to 2^-17 (bf16), 2^-22 (f16).
//
// V rows that a tile holds behind the sequence's last token are zeroed.  A row that
// comes out as NaN (a V row that another row of its tile sees may hold an infinity or
// a NaN, and 0 * V is NaN then) is computed again by exact_row.
//
// Tensor memory: S / P 2 x 128 columns, O 2 x 128.  Bound: the tensor cores.
#include "prefill_mma.cuh"
#include "tc_utils.cuh"

namespace pkv {

namespace {

constexpr int kRowsTile = 128;
constexpr int kKeys = 128;
constexpr int kThreads = 384;  // (warps 10 and 11 fill the third warpgroup and do nothing)
// Registers of a thread of the first two warpgroups and of the third: the launch's
// 168 each (65,536 over 384 threads) divided anew, 2 x 208 + 88 = 3 x 168.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr uint32_t kSlice = kKeys * 128;  // 128 rows of 64 elements: 16 KiB
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.f;

template <int D>
struct Layout {
    static constexpr uint32_t kTile = (D / 64) * kSlice;  // Q of a row tile, K or V of 128 keys
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kRing = 2 * kTile;
    static constexpr uint32_t kBars = kRing + kStages * kTile;
};

template <int kStages>
struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint32_t tmem;
    int abort;
};

// What an item needs to know, the same in every role.
struct Item {
    int s, h, ntok, pos0, ctx;
    int64_t tok0;
    int skip;    // keys between the first tokens' boxes and the window's that no row sees
    int sink_keys, boxes, tiles;
};

// Columns [lo, hi) of 32 as bits.
__device__ __forceinline__ uint32_t columns(int lo, int hi) {
    const uint32_t upto = hi <= 0 ? 0u : hi >= 32 ? 0xffffffffu : (1u << hi) - 1u;
    const uint32_t below = lo <= 0 ? 0u : lo >= 32 ? 0xffffffffu : (1u << lo) - 1u;
    return upto & ~below;
}

__device__ __forceinline__ void tensor_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                               uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// Operand descriptors (see tc_sdesc) from their low words: the high word is the
// same for every operand here (8-row groups 1024 bytes apart, 128-byte swizzle), and
// a step along an operand adds its bytes / 16 to the low one.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// 16 consecutive 32-bit columns of this warp's 32 lanes.
__device__ __forceinline__ void tc_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Two fp32 products and sums in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
          "l"(reinterpret_cast<const uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return d;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float x0, float x1) {
    if constexpr (DT == kBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x0, x1);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// kTwo: P in two parts.
template <int DT, int D, int G, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1) paged_window_prefill_tc_kernel(const PrefillArgs a,
                                                                               const __grid_constant__ CUtensorMap tmq,
                                                                               const __grid_constant__ CUtensorMap tmk,
                                                                               const __grid_constant__ CUtensorMap tmv) {
    using L = Layout<D>;
    constexpr int kStages = L::kStages;
    constexpr int kSlices = D / 64;
    constexpr int kTileTokens = kRowsTile / G;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    auto* B = reinterpret_cast<Bars<kStages>*>(base + L::kBars);
    volatile int* abort = &B->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_allow_next();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&B->full[i], 1);
            mbar_init(&B->empty[i], 1);
        }
        mbar_init(&B->q_full, 1);
        mbar_init(&B->q_empty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&B->s_full[t], 1);
            mbar_init(&B->p_full[t], 4);
            mbar_init(&B->o_full[t], 1);
        }
        B->abort = 0;
        fence_barrier_init();
        prefetch_tensor_map(&tmq);
        prefetch_tensor_map(&tmk);
        prefetch_tensor_map(&tmv);
    }
    if (warp == 9) tc_alloc(&B->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = B->tmem;
    pdl_wait();

    const int tiles = a.tile_cum[a.num_seqs];
    const int64_t items = static_cast<int64_t>(tiles) * a.num_kv_heads;
    const int box = a.box;
    const int per_tile = kKeys / box;  // boxes of a tile
    auto item_at = [&](int64_t i) {
        Item it;
        it.h = static_cast<int>(i / tiles);
        const int4* d = reinterpret_cast<const int4*>(a.tiles) + 2 * (i - static_cast<int64_t>(it.h) * tiles);
        const int4 u = d[0], v = d[1];
        it.s = u.x;
        it.tok0 = u.y;
        it.ntok = u.z;
        it.pos0 = u.w;
        it.ctx = v.x;
        const int lo = max(0, it.pos0 - a.window + 1) / box, sb = (a.sinks + box - 1) / box;
        const int skip = max(0, lo - sb);
        it.skip = skip * box;
        it.sink_keys = sb * box;
        it.boxes = (it.pos0 + it.ntok - 1) / box + 1 - skip;
        it.tiles = (it.boxes + per_tile - 1) / per_tile;
        return it;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity & 1u, abort, a.status); };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            // ---- producer
            const uint64_t keep = policy_evict_last();
            uint32_t stage = 0, round = 0, nq = 0;
            bool ok = true;
            // K or V of 128 keys: lane e issues box e / kSlices, slice e % kSlices.
            auto load = [&](const Item& it, int j, const CUtensorMap* map) -> bool {
                const int b = j * per_tile + lane / kSlices;
                const bool mine = lane < per_tile * kSlices && b < it.boxes;
                int y = 0;
                if (mine) {
                    const int cg = b * box;
                    const int key = cg + (cg >= it.sink_keys ? it.skip : 0);
                    const int lb = key / a.block_size;
                    int blk = a.block_tables[static_cast<int64_t>(it.s) * a.max_blocks + lb];
                    if (blk < 0 || blk >= a.num_blocks) {
                        raise_flag(a.status, kFlagBadBlock);
                        blk = 0;
                    }
                    y = (blk * a.num_kv_heads + it.h) * a.block_size + (key - lb * a.block_size);
                }
                int good = 1;
                if (lane == 0) {
                    if (round > 0) good = wait(&B->empty[stage], round - 1);
                    if (good) {
                        const int n = min(per_tile, it.boxes - j * per_tile);
                        mbar_arrive_expect_tx(&B->full[stage], static_cast<uint32_t>(n * box) * 128u * kSlices);
                    }
                }
                good = __shfl_sync(0xffffffffu, good, 0);
                if (!good) return false;
                if (mine) {
                    const int sl = lane % kSlices;
                    tensor_load_2d(base + L::kRing + stage * L::kTile + sl * kSlice + (lane / kSlices) * box * 128, map, sl * 64, y,
                                   &B->full[stage], keep);
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    ++round;
                }
                return true;
            };
            for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
                const Item it = item_at(i);
                const int row_tiles = it.ntok > kTileTokens ? 2 : 1;
                for (int j = 0; j < it.tiles && ok; ++j) {
                    ok = load(it, j, &tmk) && load(it, j, &tmv);
                    if (ok && j == 0) {
                        // Q, once the S of the item before are done with the buffer.
                        int good = 1;
                        if (lane == 0) {
                            if (nq > 0) good = wait(&B->q_empty, nq - 1);
                            if (good) {
                                mbar_arrive_expect_tx(&B->q_full, static_cast<uint32_t>(row_tiles) * L::kTile);
                                for (int t = 0; t < row_tiles; ++t)
                                    for (int sl = 0; sl < kSlices; ++sl)
                                        tensor_load_3d(base + L::kQ + t * L::kTile + sl * kSlice, &tmq, sl * 64, it.h * G,
                                                       static_cast<int>(it.tok0) + t * kTileTokens, &B->q_full, keep);
                                ++nq;
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                    }
                }
            }
            // Every copy issued must land before the CTA can exit.
            if (lane == 0) {
                auto drain = [&](uint64_t* bar, uint32_t parity) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(bar, parity & 1u)) {
                        if (global_timer_ns() - t0 > kWaitLimitNs) {
                            raise_flag(a.status, kFlagTimeout);
                            break;
                        }
                    }
                };
                for (uint32_t st = 0; st < kStages; ++st) {
                    const uint32_t fills = round + (st < stage ? 1u : 0u);
                    if (fills > 0) drain(&B->full[st], fills - 1);
                }
                if (nq > 0) drain(&B->q_full, nq - 1);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---- MMA issue
            if (lane == 0) {
                constexpr int bf = DT == kBF16 ? 1 : 0;
                constexpr uint32_t idS = tc_idesc_f16(bf, false, kKeys, kRowsTile);
                constexpr uint32_t idPV = tc_idesc_f16(bf, true, D, kRowsTile);
                const uint32_t qa = smem_addr(base + L::kQ), ring = smem_addr(base + L::kRing);
                uint32_t nq = 0, np[2] = {0, 0};
                uint32_t at = 0;  // ring position of the next stage to be used
                auto stage_of = [&](uint32_t x) { return x % kStages; };
                auto ready = [&](uint32_t x) { return wait(&B->full[stage_of(x)], x / kStages); };
                auto qk = [&](int t, uint32_t x) {
                    const uint32_t k = desc_low(ring + stage_of(x) * L::kTile, 16), q = desc_low(qa + t * L::kTile, 16);
    #pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t step = ((ks >> 2) * kSlice + (ks & 3) * 32) >> 4;
                        mma_ss(taddr + t * kKeys, q + step, k + step, idS, ks > 0);
                    }
                    tc_commit(&B->s_full[t]);
                };
                auto pv = [&](int t, uint32_t x, bool first) {
                    const uint32_t va = desc_low(ring + stage_of(x) * L::kTile, kSlice);
    #pragma unroll
                    for (int part = 0; part < (kTwo ? 2 : 1); ++part)
    #pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            mma_ts(taddr + 256 + t * 128, taddr + t * kKeys + part * 64 + kk * 8, va + ((kk * 16 * 128) >> 4), idPV,
                                   !(first && part == 0 && kk == 0));
                };
                bool ok = true;
                for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
                    const Item it = item_at(i);
                    const int row_tiles = it.ntok > kTileTokens ? 2 : 1;
                    ok = wait(&B->q_full, nq++) && ready(at);
                    if (!ok) break;
                    tc_fence_after();
                    for (int t = 0; t < row_tiles; ++t) qk(t, at);
                    tc_commit(&B->empty[stage_of(at)]);
                    if (it.tiles == 1) tc_commit(&B->q_empty);
                    for (int j = 0; j < it.tiles && ok; ++j) {
                        const uint32_t v = at + 1, k = at + 2;  // this tile's V, the next one's K
                        const bool more = j + 1 < it.tiles;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (t >= row_tiles || !ok) continue;
                            if (t == 0) ok = ready(v);
                            ok = ok && wait(&B->p_full[t], np[t]++);
                            if (!ok) continue;
                            tc_fence_after();
                            pv(t, v, j == 0);
                            if (t == row_tiles - 1) tc_commit(&B->empty[stage_of(v)]);
                            if (!more) {
                                tc_commit(&B->o_full[t]);
                                continue;
                            }
                            if (t == 0) ok = ready(k);
                            if (!ok) continue;
                            tc_fence_after();
                            qk(t, k);
                            if (t == row_tiles - 1) {
                                tc_commit(&B->empty[stage_of(k)]);
                                if (j + 2 == it.tiles) tc_commit(&B->q_empty);
                            }
                        }
                        at += 2;
                    }
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---- softmax: thread r of warps 4t .. 4t + 3 owns row r of row tile t
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lane_base = taddr + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t s_col = lane_base + t * kKeys, o_col = lane_base + 256 + t * 128;
        const float sc = fmaxf(fabsf(a.scale_log2), 1e-30f);  // (zero: every finite score's exponent is 0)
        const bool negative = a.scale_log2 < 0.f;
        uint32_t ns = 0, no = 0, at = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
            const Item it = item_at(i);
            const int first = t * kTileTokens;  // of this row tile, among the item's tokens
            if (first >= it.ntok) {             // (row tile 1 of a short item)
                at += 2 * it.tiles;
                continue;
            }
            const int tr = first + r / G;
            const bool mine = tr < it.ntok;
            const int qpos = it.pos0 + min(tr, it.ntok - 1);
            const int p_first = it.pos0 + first, p_last = it.pos0 + min(first + kTileTokens, it.ntok) - 1;
            // Keys in sight, as places in the list: [0, va) and [vb, vc).
            const int va = min(a.sinks, qpos + 1), vb = max(0, qpos - a.window + 1 - it.skip), vc = qpos + 1 - it.skip;
            const int all_from = max(0, p_last - a.window + 1 - it.skip), all_to = p_first + 1 - it.skip;
            const int all_sinks = min(a.sinks, p_first + 1);
            const int live = min(it.ctx - it.skip, it.boxes * box);  // places behind it hold no token
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < it.tiles; ++j, at += 2) {
                ok = __all_sync(0xffffffffu, wait(&B->s_full[t], ns++));
                if (!ok) break;
                tc_fence_after();
                float sv[kKeys];
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    float x[32];
                    tc_ld32(s_col + 32 * q4, x);
#pragma unroll
                    for (int c = 0; c < 32; ++c) sv[32 * q4 + c] = x[c];
                }
                tc_wait_ld();
                const int k0 = j * kKeys;
                if (negative) {
#pragma unroll
                    for (int c = 0; c < kKeys; ++c) sv[c] = -sv[c];
                }
                if (!((k0 >= all_from && k0 + kKeys <= all_to) || k0 + kKeys <= all_sinks)) {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        const int c0 = k0 + 32 * q4;
                        const uint32_t seen = columns(0, va - c0) | columns(vb - c0, vc - c0);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            sv[32 * q4 + c] = (seen >> c) & 1u ? sv[32 * q4 + c] : -INFINITY;
                    }
                }
                float mx[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) mx[c] = sv[c];
#pragma unroll
                for (int c = 8; c < kKeys; c += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        mx[e] = c + 8 + e < kKeys ? fmaxf(fmaxf(mx[e], sv[c + e]), sv[c + 8 + e]) : fmaxf(mx[e], sv[c + e]);
                const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                       fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) *
                                 sc;
                if (j == 0) {
                    m_ref = mt;  // -inf: nothing in sight so far
                } else {
                    const bool need = mt > m_ref + kLazy;
                    if (__any_sync(0xffffffffu, need)) {
                        const float f = need ? fast_exp2(m_ref - mt) : 1.f;  // (0 from -inf)
                        if (need) {
                            l *= f;
                            m_ref = mt;
                        }
#pragma unroll
                        for (int cb = 0; cb < D / 32; ++cb) {
                            float o[32];
                            tc_ld32(o_col + 32 * cb, o);
                            tc_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] *= f;
                            tc_st32(o_col + 32 * cb, o);
                        }
                    }
                }
                const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
                const float2 sc2 = make_float2(sc, sc), neg2 = make_float2(neg, neg);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    uint32_t hi[16];
                    [[maybe_unused]] uint32_t lo[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 e = fma2(make_float2(sv[32 * q4 + 2 * c], sv[32 * q4 + 2 * c + 1]), sc2, neg2);
                        const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                        sum[c & 1] = add2(sum[c & 1], p);
                        if constexpr (kTwo)
                            pack_split<DT>(p.x, p.y, hi[c], lo[c]);
                        else
                            hi[c] = pack2<DT>(p.x, p.y);
                    }
                    tc_st16u(s_col + 16 * q4, hi);
                    if constexpr (kTwo) tc_st16u(s_col + 64 + 16 * q4, lo);
                }
                const float2 both = add2(sum[0], sum[1]);
                l += both.x + both.y;
                if (t == 0 && k0 + kKeys > live) {
                    const uint32_t st = (at + 1) % kStages;
                    ok = __all_sync(0xffffffffu, wait(&B->full[st], (at + 1) / kStages));
                    if (!ok) break;
                    const int from = max(0, live - k0);
                    uint8_t* vd = base + L::kRing + st * L::kTile;
                    for (int e = r; e < (kKeys - from) * 8 * kSlices; e += 128) {
                        const int row = from + e / (8 * kSlices), c = e % (8 * kSlices);
                        *reinterpret_cast<uint4*>(vd + (c >> 3) * kSlice + row * 128 + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_full[t]);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait(&B->o_full[t], no++));
            if (!ok) break;
            tc_fence_after();
            const float inv = 1.f / l;
            const int64_t o0 = ((it.tok0 + tr) * a.num_q_heads + it.h * G + r % G) * D;
            bool nan = false;
#pragma unroll
            for (int cb = 0; cb < D / 32; ++cb) {
                float o[32];
                tc_ld32(o_col + 32 * cb, o);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    o[c] *= inv;
                    nan = nan || o[c] != o[c];
                }
                if (!mine) continue;
                if constexpr (kTwo) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o0 + 32 * cb);
#pragma unroll
                    for (int c = 0; c < 8; ++c) dst[c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                } else {
                    using T = typename Elem<DT>::T;
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + o0 + 32 * cb);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        dst[c] = make_uint4(pack2<DT>(o[8 * c], o[8 * c + 1]), pack2<DT>(o[8 * c + 2], o[8 * c + 3]),
                                            pack2<DT>(o[8 * c + 4], o[8 * c + 5]), pack2<DT>(o[8 * c + 6], o[8 * c + 7]));
                }
            }
            tc_fence_before();  // O is read before this thread lets the next P . V begin
            uint32_t bad = __ballot_sync(0xffffffffu, nan && mine);
            __syncwarp();
            for (; bad; bad &= bad - 1) {
                const int row = first * G + (warp & 3) * 32 + __ffs(bad) - 1;
                exact_row<DT, DT, D>(a, it.s, it.h, it.tok0 + row / G, it.h * G + row % G, it.pos0 + row / G);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tc_dealloc(taddr, kTmemCols);
    }
}

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

template <int DT, int D, int G, bool kTwo>
cudaError_t launch_tc(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int ctas,
                      cudaStream_t stream) {
    static RaisedLimit limit;
    auto kern = paged_window_prefill_tc_kernel<DT, D, G, kTwo>;
    const cudaError_t e = allow_shared_memory(kern, a.device, a.smem_bytes, &limit);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(ctas), dim3(kThreads), static_cast<size_t>(a.smem_bytes), stream, a.pdl != 0, a, tmq, tmk,
                         tmv);
}

template <int DT, int D, bool kTwo>
cudaError_t launch_tc_g(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int ctas,
                        cudaStream_t stream) {
    switch (a.num_q_heads / a.num_kv_heads) {
        case 1: return launch_tc<DT, D, 1, kTwo>(a, tmq, tmk, tmv, ctas, stream);
        case 2: return launch_tc<DT, D, 2, kTwo>(a, tmq, tmk, tmv, ctas, stream);
        case 4: return launch_tc<DT, D, 4, kTwo>(a, tmq, tmk, tmv, ctas, stream);
        case 8: return launch_tc<DT, D, 8, kTwo>(a, tmq, tmk, tmv, ctas, stream);
    }
    return cudaErrorInvalidValue;
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
    return head_dim == 128 ? static_cast<int>(Layout<128>::kBars + sizeof(Bars<Layout<128>::kStages>)) + 1024
                           : static_cast<int>(Layout<64>::kBars + sizeof(Bars<Layout<64>::kStages>)) + 1024;
}

cudaError_t launch_window_prefill_tc(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk,
                                     const CUtensorMap& tmv, int num_sms, cudaStream_t stream) {
    const cudaError_t e = launch_kernel(window_prefill_plan_kernel, dim3(1), dim3(1024), 0, stream, a.pdl != 0, a);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(a.grid_tiles) * a.num_kv_heads;
    const int ctas = static_cast<int>(items < num_sms ? items : num_sms);
    if (a.dtype == kBF16) return launch_tc_t<kBF16>(a, tmq, tmk, tmv, ctas, stream);
    if (a.dtype == kF16) return launch_tc_t<kF16>(a, tmq, tmk, tmv, ctas, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
