// Decode attention of a batch in which groups of sequences share the blocks
// of a long prefix ("Reading Inference Engine Codebases", Examples 12 and 13:
// requests with equal prompts are given the same cached blocks): each group's
// prefix is read once for all its members.
//
// The mathematics.  For one query row, softmax over a set of keys cut into
// parts needs of each part only m = max score (or any reference), l = sum of
// 2^(score - m) and O = sum of 2^(score - m) V; the whole is
// sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  A group's prefix is
// attended to by all members alike, without a mask, so its scores are one
// matrix product per KV head: rows = (member, query head of the KV head),
// columns = prefix keys.  What follows the prefix differs per sequence and is
// left to the split-context decode kernel's code.  Two launches:
//   attend  one CTA an SM, in one of two roles that run side by side:
//             parts  (m, l, O) of 128 rows over a range of a group's keys;
//             tails  the decode kernel over the tokens after the prefix,
//                    partials only;
//   merge   one warp a (sequence, query head).
// Which sequences share (those at least as long as the prefix; shorter ones
// read their own tables throughout) and how the work is cut follows from the
// groups and lengths alone, so every CTA works it out for itself
// (prefix_units.cuh), which costs less than a launch that does it for all.
//
// The parts role.  Producer warps bring K and V tiles of 64 keys into swizzled
// shared memory; two warps issue tcgen05 MMAs, S = Q K^T into tensor memory
// (four buffers) and O += P V with P read from tensor memory; two groups of
// four warps hold the softmax, one row a thread.  Tiles alternate between the
// two groups (and issuers), each with an accumulator of its own: a group's
// softmax of a tile takes about 1 us, mostly latency, and an issuing warp
// whose sub-partition also runs softmax warps issues an MMA only every 100
// cycles or so, where the tensor pipe takes 64; two of each keep it busy.
// (Measured on 256 sequences, 32 query and 8 KV heads, 32,768 shared tokens:
// 356 us with one issuing lane, 290 with one warp walking the issue loop
// converged, so that descriptors stay in uniform registers, 214 with two.)
// P enters the product as a high and a low half-precision part, 1.5 times the
// matrix work of one part, whose rounding (2^-9 of each weight in bf16) would
// be as large as that of a bf16 output.  Two bf16 parts hold a weight to 2^-17
// of it.  Two f16 parts hold it to 2^-22, but nothing below half of f16's
// smallest step: the reference lies weight_shift below the score that it stands
// for, so that what a weight loses there is at most 2^-32 of the largest.
//
// The sums in tensor memory are fp32, but each step of them drops what lies past
// the last place, so that a long sum of one sign comes out low: with V = 1 and 256
// sequences of 32 query and 8 KV heads, 1.3e-6 over 4,096 shared tokens (bf16),
// 9.6e-6 over 32,768 and 4.1e-5 over 131,072; up to twice that in f16, 4.1e-4 (half
// a step of an f16 output is 4.9e-4) over 524,288.  The decode kernel's warp MMAs
// do the same (f16, 524,288 tokens: 4.3e-4).
//
// Bounds and measurements (128-dim heads, 32 query and 8 KV heads, bf16, both
// launches, calls in a graph; after 256 MB of other reads in brackets, which is
// how a layer finds a cache that the layers before it have put out of L2):
// - up to 128 query rows a KV head: the memory, and below some 10 us the start
//   of the roles, one after another latency, and the merge (32 sequences,
//   4,096 shared tokens: 22 us [36]; 65,536 shared: 66 us [70], 4.1 TB/s of K
//   and V);
// - more: the tensor pipe, 50 % active by its counter (256 sequences, 32,768
//   shared: 188 us [191], 740 TFLOP/s, or 1,110 of matrix work).
// Registers: 168 a thread over 16-bit caches, with 68 bytes of spill stores (32
// with 64 dims); 128 a thread over E4M3, with 344 to 364.
// Tried and left: 2 KB tensor copies for K and V (61 ns each on one SM, slower
// than 16-byte copies by 10 % where matrix work bounds), one softmax group a CTA
// with two CTAs an SM (219 us on the wide case, and no room for tails beside
// it), packed fp32 pairs in the softmax (-5 % on the wide case, +3 % on small).
#pragma once

#include "decode_kernel.cuh"
#include "mma_frag.cuh"
#include "shared_prefix.cuh"
#include "tc_utils.cuh"

namespace pkv {

namespace {

constexpr int kBM = kPrefixRows;
constexpr int kNK = kPrefixTile;
constexpr int kS = 4;                // S / P buffers in tensor memory, 64 columns each
constexpr uint32_t kO = kS * kNK;    // the two accumulators, D columns each
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.f;  // a row's scores may pass its reference by this much (log2) before the sums are rescaled
// log2 of a weight at the reference: the f16 parts' range is used up to 2^(kLazy + 7) = 2^15.
__host__ __device__ constexpr float weight_shift(int dt) { return dt == static_cast<int>(kF16) ? 7.f : 0.f; }
constexpr int kSoftmaxWarps = 8;
// E4M3: codes on their way to be widened, tiles a producer warp.
constexpr int kRawRing = 5;
// Producer warps of K and of V: an E4M3 tile is widened by two of each.
__host__ __device__ constexpr int producers(bool fp8) { return fp8 ? 2 : 1; }
__host__ __device__ constexpr int parts_threads(bool fp8) { return 32 * (kSoftmaxWarps + 2 + 2 * producers(fp8)); }

template <int D, bool kFP8>
struct Shape {
    static constexpr int kSlices = D / 64;                    // 128-byte slices of a row
    static constexpr int kKRing = kFP8 ? 3 : D == 128 ? 6 : 10;  // K stages
    static constexpr int kVRing = kFP8 ? 3 : D == 128 ? 5 : 10;  // V stages
    static constexpr uint32_t kTile = kSlices * kNK * 128;    // bytes of a K (or V) tile
    static constexpr uint32_t kQOff = 0;
    static constexpr uint32_t kKOff = kSlices * kBM * 128;
    static constexpr uint32_t kVOff = kKOff + kKRing * kTile;
    static constexpr uint32_t kRawOff = kVOff + kVRing * kTile;
    static constexpr uint32_t kBytes = kRawOff + (kFP8 ? 2 * kRawRing * kNK * 128 : 0);
};

struct Bars {
    uint64_t kfull[10], kempty[10], vfull[10], vempty[10];
    uint64_t s_full[kS], p_full[kS], pv_done[kS], tmem_ready;
    uint64_t q_full[2];  // segments in turn: an issuing warp without a tile in one may be a segment late
    float2 ml[2][kBM];  // (reference, sum) of each row in each softmax group
    float down[kBM];    // E4M3 with a bf16 q: what undoes each row's power of two
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
    return mbar_wait_bounded(bar, parity & 1u, abort, status);
}

// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// 32 bytes to global memory (a whole sector at once).
__device__ __forceinline__ void store_32(float* p, const float* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
                 "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])),
                 "r"(__float_as_uint(v[7]))
                 : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

// tc_mma, tc_mma_ts and tc_commit issued by the lane with leader != 0 while the
// whole warp walks the loop: addresses and descriptors are then the same on
// every lane, and the compiler can keep them in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi,
                                       uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t blo, uint32_t hi,
                                       uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}

// Eight E4M3 codes -> eight f16 values, exactly.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
    return make_uint4(e4m3x2_to_half2(static_cast<uint16_t>(lo)), e4m3x2_to_half2(static_cast<uint16_t>(lo >> 16)),
                      e4m3x2_to_half2(static_cast<uint16_t>(hi)), e4m3x2_to_half2(static_cast<uint16_t>(hi >> 16)));
}

// QT: q's type.  The tensor cores work in it, or in f16 over an E4M3 cache
// (whose values all are f16); a bf16 q is then brought to f16 with a power of
// two for each row that puts its largest element at 2^13: exact down to 2^-30
// of that element (f16's steps of 2^-24 hold a bf16's eight bits from 2^-17 on).

// One thread, before the roles are known.
template <int D, bool kFP8>
__device__ __forceinline__ void init_bars(Bars* B) {
    using S = Shape<D, kFP8>;
    // A tile is full with one arrival of each of its producer warps, or one a copying lane.
    for (int i = 0; i < S::kKRing; ++i) {
        mbar_init(&B->kfull[i], kFP8 ? producers(true) : 32);
        mbar_init(&B->kempty[i], 1);
    }
    for (int i = 0; i < S::kVRing; ++i) {
        mbar_init(&B->vfull[i], kFP8 ? producers(true) : 32);
        mbar_init(&B->vempty[i], 1);
    }
    for (int i = 0; i < kS; ++i) {
        mbar_init(&B->s_full[i], 1);
        mbar_init(&B->p_full[i], 4);
        mbar_init(&B->pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&B->q_full[i], kSoftmaxWarps);
    mbar_init(&B->tmem_ready, 1);
    B->abort = 0;
    fence_barrier_init();
}

template <int QT, int D, bool kFP8>
__device__ __forceinline__ void parts_cta(const SharedPrefixArgs& a, uint8_t* base, Bars* B, const Units& units, int cta) {
    using T = typename Elem<QT>::T;
    using S = Shape<D, kFP8>;
    constexpr int DT = kFP8 ? static_cast<int>(kF16) : QT;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.num_q_heads / a.num_kv_heads;
    const int start = mul_div(cta, units.W, units.P), end = mul_div(cta + 1, units.W, units.P);
    volatile int* abort = &B->abort;
    // All of tensor memory is taken, so its addresses start at 0.
    constexpr uint32_t taddr = 0;

    // Every role walks the CTA's segments; tiles are counted from the CTA's
    // first (i), so rings and buffers go on over segments.
    if (warp >= kSoftmaxWarps + 2) {
        // ---- producers.  The keys come in runs of 16 rows (block_size is a
        // multiple of 16), each inside one block; runs past the last key are
        // zeros.
        const int bs = a.block_size;
        const int ch = lane & 7, l8 = lane >> 3;
        const int w = (warp - kSoftmaxWarps - 2) & 1;  // 0: K tiles, 1: V tiles
        const char* cache = static_cast<const char*>(w == 0 ? a.k_cache : a.v_cache);
        uint8_t* tiles = base + (w == 0 ? S::kKOff : S::kVOff);
        uint64_t* full = w == 0 ? B->kfull : B->vfull;
        uint64_t* empty = w == 0 ? B->kempty : B->vempty;
        const int ring = w == 0 ? S::kKRing : S::kVRing;
        int i = 0;  // tiles before the segment
        bool ok = true;
        for (int x = start; x < end && ok;) {
            const Triple t = find_triple(a, units, G, x);
            const int n = min(end, t.tile0 + t.keys) - x;  // tiles of the segment
            const int key0 = (x - t.tile0) * kNK;
            const int nruns = (min(t.blocks * bs, key0 + n * kNK) - key0) / 16;
            // The member whose table row names the blocks; without one the
            // segment's keys are zeros and nobody reads its part.
            int lead = -1;
            for (int s0 = 0; s0 * G < t.rows && lead < 0; s0 += 32) {
                const int s = t.seq0 + s0 + lane;
                const uint32_t in = __ballot_sync(0xffffffffu, (s0 + lane) * G < t.rows && a.context_lens[s] / bs >= t.blocks);
                if (in) lead = t.seq0 + s0 + __ffs(in) - 1;
            }
            const int32_t* table = a.block_tables + static_cast<int64_t>(lead < 0 ? 0 : lead) * a.max_blocks;
            // First cache row of run r of the segment; -1: zeros.
            auto run_row = [&](int r) -> int {
                if (r >= nruns || lead < 0) return -1;
                const int key = key0 + 16 * r;
                const int lb = key / bs;
                int blk = table[lb];
                if (blk < 0 || blk >= a.num_blocks) {
                    raise_flag(a.status, kFlagBadBlock);
                    blk = 0;
                }
                return (blk * a.num_kv_heads + t.h) * bs + (key - lb * bs);
            };
            // Lane l knows where run l of the current 8 tiles starts, and of the 8
            // after them; lane e takes the 16 bytes e % 8 of rows e / 8 + 4 q of a
            // run (of both 64-element slices).
            int now = run_row(lane), next = run_row(32 + lane);
            auto advance = [&](int j) {  // to tile j
                if ((j & 7) == 0 && j > 0) {
                    now = next;
                    next = run_row(4 * (j + 8) + lane);
                }
            };
            int st = i % ring, round = i / ring;
            auto vacant = [&]() {
                return round == 0 || __all_sync(0xffffffffu, wait(&empty[st], round - 1, abort, a.status)) != 0;
            };
            if constexpr (!kFP8) {
                const char* c0 = cache + l8 * (D * 2) + ch * 16;
                const uint32_t d0 = smem_addr(tiles) + l8 * 128;
                const uint32_t sw0 = static_cast<uint32_t>(ch ^ l8) << 4, sw1 = static_cast<uint32_t>(ch ^ (l8 + 4)) << 4;
                for (int j = 0; j < n; ++j) {
                    advance(j);
                    ok = vacant();
                    if (!ok) break;
                    const uint32_t dst = d0 + st * S::kTile;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = __shfl_sync(0xffffffffu, now, (j & 7) * 4 + k);
                        const bool real = row >= 0;
                        const char* src = c0 + (real ? static_cast<int64_t>(row) * (D * 2) : 0);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t d = dst + (16 * k + 4 * q) * 128 + ((q & 1) ? sw1 : sw0);
#pragma unroll
                            for (int sl = 0; sl < S::kSlices; ++sl)
                                cp_async_16_or_zero(d + sl * (kNK * 128), src + (real ? q * (4 * D * 2) + sl * 128 : 0), real);
                        }
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&full[st])) : "memory");
                    if (++st == ring) st = 0, ++round;
                }
            } else {
                // E4M3: the codes travel through a ring of this warp's own (each
                // lane reads back what it copied) and are widened into its
                // share of the tile's runs; lane e takes codes 16 (e % 8) .. of a
                // row.
                constexpr int kRuns = 4 / producers(true);
                constexpr uint32_t kStage = kRuns * 16 * 128;
                const int share = (warp - kSoftmaxWarps - 2) >> 1;
                const char* c0 = cache + l8 * D + ch * 16;
                const uint32_t raw0 = smem_addr(base + S::kRawOff) + (share * 2 + w) * (kRawRing * kStage) + lane * 16;
                auto ask = [&](int j) {  // in order; an empty group past the end
                    if (j < n) {
                        advance(j);
                        const uint32_t d = raw0 + j % kRawRing * kStage;
#pragma unroll
                        for (int k = 0; k < kRuns; ++k) {
                            const int row = __shfl_sync(0xffffffffu, now, (j & 7) * 4 + share * kRuns + k);
                            const bool real = row >= 0;
                            const char* src = c0 + (real ? static_cast<int64_t>(row) * D : 0);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                cp_async_16_or_zero(d + (4 * k + q) * 512, src + (real ? 4 * q * D : 0), real);
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                for (int j = 0; j < kRawRing - 1; ++j) ask(j);
                for (int j = 0; j < n; ++j) {
                    ask(j + kRawRing - 1);
                    asm volatile("cp.async.wait_group %0;" ::"n"(kRawRing - 1) : "memory");  // tile j is here
                    const uint32_t raw = raw0 + j % kRawRing * kStage;
                    uint8_t* t0 = tiles + st * S::kTile + (ch >> 2) * (kNK * 128);
                    uint4 r[4 * kRuns];
#pragma unroll
                    for (int q = 0; q < 4 * kRuns; ++q)
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(r[q].x), "=r"(r[q].y), "=r"(r[q].z), "=r"(r[q].w)
                                     : "r"(raw + q * 512));
                    ok = vacant();
                    if (!ok) break;
#pragma unroll
                    for (int q = 0; q < 4 * kRuns; ++q) {
                        const int row = 16 * kRuns * share + 4 * q + l8;
                        const int c2 = (ch & 3) * 2;
                        *reinterpret_cast<uint4*>(t0 + row * 128 + ((c2 ^ (row & 7)) << 4)) = widen8(r[q].x, r[q].y);
                        *reinterpret_cast<uint4*>(t0 + row * 128 + (((c2 + 1) ^ (row & 7)) << 4)) = widen8(r[q].z, r[q].w);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[st]);
                    if (++st == ring) st = 0, ++round;
                }
            }
            i += n;
            x += n;
        }
        // Every copy issued must land before the CTA can exit.
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp >= kSoftmaxWarps) {
        // ---- MMA issue: each of two warps issues for the tiles of one parity,
        // S one of them ahead of P V.
        constexpr int bf = DT == kBF16 ? 1 : 0;
        constexpr uint32_t idS = tc_idesc_f16(bf, false, kNK, kBM);
        constexpr uint32_t idPV = tc_idesc_f16(bf, true, D, kBM);
        const int me = warp - kSoftmaxWarps;
        const uint32_t leader = elect_one();
        const uint32_t sbase = smem_addr(base), bars = smem_addr(B);
        auto bar_of = [&](const uint64_t* p) { return bars + static_cast<uint32_t>(reinterpret_cast<const uint8_t*>(p) - reinterpret_cast<const uint8_t*>(B)); };
        // Descriptors: the low word holds the address and the slice distance, the
        // high word (the row groups' distance) is the same for all.
        constexpr uint32_t kHi = static_cast<uint32_t>((1024u >> 4) | (1u << 14) | (2u << 29));
        const uint32_t qd = ((sbase + S::kQOff) >> 4) | (1u << 16);
        auto ready = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, wait(bar, phase, abort, a.status)) != 0; };
        auto score = [&](int i) -> bool {
            const int sk = i % S::kKRing, b = i % kS;
            if (!ready(&B->kfull[sk], i / S::kKRing)) return false;
            // S buffer b holds P of tile i - kS until that PV has completed.
            if (i >= kS && !ready(&B->pv_done[b], i / kS - 1)) return false;
            if constexpr (!kFP8) fence_proxy_async_smem();  // lane copies before the tensor cores read them
            tc_fence_after();
            const uint32_t kd = ((sbase + S::kKOff + sk * S::kTile) >> 4) | (1u << 16);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_ss(leader, b * kNK, qd + (((ks >> 2) * (kBM * 128) + (ks & 3) * 32) >> 4),
                       kd + (((ks >> 2) * (kNK * 128) + (ks & 3) * 32) >> 4), kHi, idS, ks > 0);
            mma_commit(leader, bar_of(&B->s_full[b]));
            mma_commit(leader, bar_of(&B->kempty[sk]));
            return true;
        };
        auto pv = [&](int i, bool first) -> bool {
            const int sv = i % S::kVRing, b = i % kS;
            if (!ready(&B->p_full[b], i / kS)) return false;
            if (!ready(&B->vfull[sv], i / S::kVRing)) return false;
            if constexpr (!kFP8) fence_proxy_async_smem();
            tc_fence_after();
            const uint32_t vd = ((sbase + S::kVOff + sv * S::kTile) >> 4) | ((kNK * 128 >> 4) << 16);
            const uint32_t o = kO + (i & 1) * D;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < kNK / 16; ++kk)
                    mma_ts(leader, o, b * kNK + part * 32 + kk * 8, vd + ((kk * 16 * 128) >> 4), kHi, idPV,
                           !(first && part == 0 && kk == 0));
            mma_commit(leader, bar_of(&B->pv_done[b]));
            mma_commit(leader, bar_of(&B->vempty[sv]));
            return true;
        };
        int i = 0, seg = 0;
        bool ok = true;
        if (me == 0) {
            tc_alloc(&B->tmem, kTmemCols);
            tc_fence_before();
            if (lane == 0) mbar_arrive(&B->tmem_ready);
            __syncwarp();
        } else {
            ok = ready(&B->tmem_ready, 0);
            tc_fence_after();
        }
        for (int x = start; x < end && ok; ++seg) {
            const Triple t = find_triple(a, units, G, x);
            const int n = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(min(end, t.tile0 + t.keys) - x)));
            const int j0 = (me ^ i) & 1;
            ok = ready(&B->q_full[seg & 1], seg >> 1);
            if (ok && j0 < n) ok = score(i + j0);
            for (int j = j0; j < n && ok; j += 2) {
                if (j + 2 < n) ok = score(i + j + 2);
                if (ok) ok = pv(i + j, j < 2);
            }
            i += n;
            x += n;
        }
    } else {
        // ---- softmax: two groups of four warps; group g takes the tiles whose
        // count has parity g, with a reference, a sum and an accumulator of its
        // own.  Thread r of a group owns row r (tensor-memory lane r).
        const int r = tid & (kBM - 1), grp = tid / kBM;
        const uint32_t lane_base = taddr + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t o_base = lane_base + kO + grp * D;
        // |scale| in log2 units; a zero multiplier is taken as 1e-30, which leaves
        // every finite score's exponent at 0 while masked scores stay -inf.
        constexpr float kLeast = 1e-30f;
        const float sc0 = fmaxf(fabsf(a.scale_log2), kLeast);
        constexpr float kUp = weight_shift(DT);
        int i = 0, seg = 0;
        bool ok = true;  // (a failed wait skips the work, not the barriers)
        for (int x = start; x < end; ++seg) {
            const Triple t = find_triple(a, units, G, x);
            const int n = min(end, t.tile0 + t.keys) - x;
            const int nrows = min(kBM, t.rows - t.rt * kBM);
            const int keys = min(t.blocks * a.block_size - (x - t.tile0) * kNK, n * kNK);  // of the segment
            {
                // Q rows of the tile (row r: member (rt * 128 + r) / G, query head
                // h * G + r % G) into shared memory, 128-byte swizzled K-major:
                // 16 rows a warp, whole rows at a time.  (The previous segment's S
                // are complete: all were read before its barriers.)
                constexpr int kChunks = D / 8, kRowsAtOnce = 32 / kChunks, kLoads = 16 / kRowsAtOnce;
                const int chunk = lane % kChunks, sub = lane / kChunks;
                // A negative scale is applied as |scale| to the scores of -q (a
                // sign flip is exact), so the row maximum is taken on unscaled
                // scores.
                const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
                uint4 q[kLoads];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int rr = t.rt * kBM + min(warp * 16 + k * kRowsAtOnce + sub, nrows - 1);
                    q[k] = *reinterpret_cast<const uint4*>(
                        static_cast<const T*>(a.q) +
                        (static_cast<int64_t>(t.seq0 + rr / G) * a.num_q_heads + t.h * G + rr % G) * D + 8 * chunk);
                }
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int row = warp * 16 + k * kRowsAtOnce + sub;
                    uint4 v = q[k];
                    if constexpr (kFP8 && QT == kBF16) {
                        uint32_t* b = &v.x;
                        uint32_t top = 0;  // the row's largest |q|, as the bits of a bf16
#pragma unroll
                        for (int c = 0; c < 4; ++c) top = max(top, max(b[c] & 0x7FFFu, (b[c] >> 16) & 0x7FFFu));
#pragma unroll
                        for (int o = 1; o < kChunks; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int e = min(max(static_cast<int>(top >> 7) - 127, -100), 127);  // its exponent
                        const float up = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
                        if (chunk == 0) B->down[row] = __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const __half2 h = __floats2half2_rn(__uint_as_float(b[c] << 16) * up,
                                                                __uint_as_float(b[c] & 0xFFFF0000u) * up);
                            b[c] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
                    v.x ^= flip;
                    v.y ^= flip;
                    v.z ^= flip;
                    v.w ^= flip;
                    *reinterpret_cast<uint4*>(base + S::kQOff + (chunk >> 3) * (kBM * 128) + row * 128 +
                                              (((chunk & 7) ^ (row & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->q_full[seg & 1]);  // one arrival per warp (count 8)
                // The CTA with a triple's first tile says where its parts are,
                // for the members of the row tile.
                const int rr = t.rt * kBM + r, s = t.seq0 + rr / G;
                if (x == t.tile0 && grp == 0 && r < nrows && rr % G == 0 && a.context_lens[s] / a.block_size >= t.blocks)
                    a.parts[static_cast<int64_t>(s) * a.num_kv_heads + t.h] =
                        make_int4(t.row0 + r, t.rows, cta_of_tile(t.tile0 + t.keys - 1, units.W, units.P) - cta + 1, 0);
            }
            // Unless it has a tile, a group weighs nothing.
            float m_ref = -1e30f, l = 0.f;
            const int j0 = (grp ^ i) & 1;
            const bool idle = 32 * (warp & 3) >= nrows;  // none of the warp's rows is anybody's: P stays as it is
            for (int j = j0; j < n && ok; j += 2) {
                const int k0 = i + j, b = k0 % kS;
                ok = __all_sync(0xffffffffu, wait(&B->s_full[b], k0 / kS, abort, a.status));
                if (!ok) break;
                if (idle) {
                    if (lane == 0) mbar_arrive(&B->p_full[b]);
                    continue;
                }
                tc_fence_after();
                float sc = sc0;
                // (down was written before the S that has come.  The product may
                // underflow to 0, and the scores over codes are below 2^14 * 448 *
                // 128 < 2^30: kLeast leaves their exponents at 0 as well.)
                if constexpr (kFP8 && QT == kBF16) sc = fmaxf(sc * B->down[r], kLeast);
                float sv[kNK];
                {
                    float t0[32], t1[32];
                    tc_ld32(lane_base + b * kNK, t0);
                    tc_ld32(lane_base + b * kNK + 32, t1);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        sv[k] = t0[k];
                        sv[32 + k] = t1[k];
                    }
                }
                const int left = keys - j * kNK;  // keys from this tile on
                if (left < kNK) {
#pragma unroll
                    for (int k = 0; k < kNK; ++k) sv[k] = k < left ? sv[k] : -INFINITY;
                }
                // Row maximum as eight independent chains (short dependency path).
                float mx[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mx[k] = fmaxf(sv[k], sv[8 + k]);
#pragma unroll
                for (int k = 16; k < kNK; k += 16)
#pragma unroll
                    for (int c = 0; c < 8; ++c) mx[c] = max3(mx[c], sv[k + c], sv[k + 8 + c]);
                // (The lower limit keeps the exponents of a row whose scores
                // are all -inf so far at -inf, not NaN.)
                const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                const float mt = fmaxf(top * sc, -1e30f) - kUp;
                bool need = false;
                if (j < 2)
                    m_ref = mt;
                else  // the largest exponent, as the weights' below: no weight passes 2^(kLazy + kUp)
                    need = fmaf(top, sc, -m_ref) > kLazy + kUp;
                if (__any_sync(0xffffffffu, need)) {
                    // O must be complete up to the group's tile before it is rescaled.
                    ok = __all_sync(0xffffffffu, wait(&B->pv_done[(k0 - 2) % kS], (k0 - 2) / kS, abort, a.status));
                    if (!ok) break;
                    tc_fence_after();
                    const float f = need ? fast_exp2(m_ref - mt) : 1.f;
                    if (need) {
                        l *= f;
                        m_ref = mt;
                    }
#pragma unroll
                    for (int cb = 0; cb < D / 32; ++cb) {
                        float o[32];
                        tc_ld32(o_base + 32 * cb, o);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= f;
                        tc_st32(o_base + 32 * cb, o);
                    }
                    tc_wait_st();
                }
                // P over the S buffer it came from: columns 0-31 the high part,
                // 32-63 the low part, keys 2k and 2k + 1 in column k.
                float ps[4] = {0.f, 0.f, 0.f, 0.f};
                {
                    uint32_t ph[32], pl[32];
#pragma unroll
                    for (int k = 0; k < kNK / 2; ++k) {
                        const float p0 = fast_exp2(fmaf(sv[2 * k], sc, -m_ref));
                        const float p1 = fast_exp2(fmaf(sv[2 * k + 1], sc, -m_ref));
                        ps[k & 3] += p0 + p1;
                        pack_split<DT>(p0, p1, ph[k], pl[k]);
                    }
                    tc_st32u(lane_base + b * kNK, ph);
                    tc_st32u(lane_base + b * kNK + 32, pl);
                }
                l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_full[b]);  // one arrival per warp (count 4)
            }
            i += n;
            // Both groups' accumulators into one part: group g writes half of
            // the columns.
            B->ml[grp][r] = make_float2(m_ref, l);
            named_barrier_sync(1, 2 * kBM);
            if (ok) ok = __all_sync(0xffffffffu, wait(&B->pv_done[(i - 1) % kS], (i - 1) / kS, abort, a.status));
            if (ok && n > 1) ok = __all_sync(0xffffffffu, wait(&B->pv_done[(i - 2) % kS], (i - 2) / kS, abort, a.status));
            if (ok) {
                tc_fence_after();
                const float2 e = B->ml[0][r], o = B->ml[1][r];
                const float M = fmaxf(e.x, o.x);
                const float we = fast_exp2(e.x - M), wo = fast_exp2(o.x - M);
                const float vs = a.v_scale;
                const float se = we * vs, so = wo * vs;
                // A segment of one tile leaves the other group's accumulator as it was.
                const bool has_e = n > 1 || ((i - 1) & 1) == 0, has_o = n > 1 || ((i - 1) & 1) == 1;
                const int64_t row = t.row0 + static_cast<int64_t>(cta - cta_of_tile(t.tile0, units.W, units.P)) * t.rows + r;
                const bool row_ok = r < nrows && row < a.max_rows;
                float* po = a.part_o + row * D + grp * (D / 2);
#pragma unroll
                for (int cb = 0; cb < D / 64; ++cb) {
                    float v0[32], v1[32];
                    tc_ld32(lane_base + kO + grp * (D / 2) + 32 * cb, v0);
                    tc_ld32(lane_base + kO + D + grp * (D / 2) + 32 * cb, v1);
                    tc_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v0[k] = (has_e ? v0[k] * se : 0.f) + (has_o ? v1[k] * so : 0.f);
#pragma unroll
                        for (int k = 0; k < 32; k += 8) store_32(po + 32 * cb + k, v0 + k);
                    }
                }
                if (row_ok && grp == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * row) = make_float2(M, we * e.y + wo * o.y);
                tc_fence_before();
            }
            named_barrier_sync(1, 2 * kBM);  // both accumulators read before the next segment's P is announced
            x += n;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftmaxWarps) {
        tc_fence_after();
        tc_dealloc(taddr, kTmemCols);
    }
}

// CTAs first .. are tails, the others parts (see decode_tails).
template <class Policy, int QT, int D, bool kFP8>
__global__ void __launch_bounds__(parts_threads(kFP8), 1)
    shared_prefix_attend_kernel(const __grid_constant__ SharedPrefixArgs a, const __grid_constant__ TailArgs d,
                                const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    static_assert(Policy::kMaxThreads == parts_threads(kFP8) && !Policy::kScratch);
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;  // of the parts role
    if (threadIdx.x == 0) init_bars<D, kFP8>(&bars);
    pdl_allow_next();
    pdl_wait();
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Units units;
    bool parts = false;
    decode_tails<Policy>(d, tmk, tmv, base, &units, &parts);
    if (!parts) return;
    parts_cta<QT, D, kFP8>(a, base, &bars, units, static_cast<int>(blockIdx.x) - (d.num_ctas - units.P));
}

template <class Policy, int QT, int D, bool kFP8>
cudaError_t launch_attend_t(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmk,
                            const CUtensorMap& tmv, cudaStream_t stream) {
    static RaisedLimit limit, carveout;
    auto kern = shared_prefix_attend_kernel<Policy, QT, D, kFP8>;
    cudaError_t e = allow_shared_memory(kern, d.device, d.smem_bytes, &limit);
    if (e == cudaSuccess) e = prefer_shared_memory(kern, d.device, &carveout);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(d.num_ctas), dim3(parts_threads(kFP8)), static_cast<size_t>(d.smem_bytes), stream, true,
                         a, d, tmk, tmv);
}

}  // namespace

}  // namespace pkv
