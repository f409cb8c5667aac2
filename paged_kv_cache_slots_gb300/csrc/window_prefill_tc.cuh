// Chunks of new tokens under a sliding window on the fifth-generation tensor cores
// (tcgen05): f16 and bf16 caches (see paged_window_prefill_attention).
//
// For a row (new token at position p, query head g) over the keys j in sight,
// j <= p and (j > p - window or j < sinks):
//   s_j = scale q . k_j,  m = max s_j,  out = sum 2^(s_j - m) v_j / sum 2^(s_j - m)
// in base 2, with one pass over the keys.  Instead of m there stands a reference that
// moves seldom: it is the maximum of the first keys that the row sees (f16: 7 below
// it, see kLower), and that of later ones when the weights of 64 keys sum to more than
// kMoveAt (O and the sum are rescaled then), so that the usual 64 keys need no maximum
// at all.
//
// Work split.  An item is 256 / G new tokens of one sequence with the G query heads
// of one KV head: 256 rows, two tiles of 128, so that a K and V tile read from L2
// serves 256 rows (at 128 rows a CTA the tensor cores would ask L2 for twice as much
// as it gives).  A persistent CTA for each SM walks its items; the keys of an item
// are a list of boxes of 16 or 32 rows of a cached block (those of the first tokens,
// then those of the window), taken 128 keys at a time:
//   warp 8       producer: Q, K and V by TMA into a Q buffer and a ring of stages
//                (a stage is the K or the V of 128 keys), ahead into the next item;
//   warp 9       issues the MMAs: S = Q . K^T of one row tile (M 128, N 128) while the
//                other's softmax runs, then O += P . V with P read from tensor memory
//                over the S it came from (an issuing warp for each row tile: the long
//                chunk 997 us instead of 888);
//   warps 0-3, 4-7  softmax of the two row tiles, a thread a row: load S, mask (the
//                tiles at the edges of the window alone), maximum, weights, P; at the
//                end of an item O / l.
// The MMAs run in the order of their issue, so that S of the next keys being there
// says that P . V of these is done: the rescaling of O needs no wait of its own.
//
// Roundings.  S, O, the maxima and sums are fp32.  With a 16-bit output a weight
// meets V rounded to q's type (half a step: as much as the output's own rounding),
// with an fp32 output in two parts, which hold it to 2^-17 (bf16), 2^-22 (f16).  f16 parts
// end at 2^-24, where the row's largest weight is 2^7 at least: a weight loses up to 2^-32
// of the largest besides.
//
// V rows that a tile holds behind the sequence's last token are zeroed.  A row that
// comes out as NaN (a V row that another row of its tile sees may hold an infinity or
// a NaN, and 0 * V is NaN then) is computed again by exact_row, once the CTA's items are
// done: a row takes 9 us for each 32 keys in sight (128 dims), and the other roles' waits,
// which give up after two seconds, must not span that.
//
// Tensor memory: S / P 2 x 128 columns, O 2 x 128.  Registers: 168 a thread as launched,
// 208 in the softmax warps.  With a 16-bit output nothing spills at 128 dims (64: 52 bytes);
// with an fp32 one 12 bytes are stored and 36 to 124 loaded, over E4M3 16 and 104.
// Bound: the tensor cores, 61 % of whose cycles it uses on long windows; the rest is the
// softmax of a tile, the issuing warp's looks at its barriers, and at short windows the
// ends of the items.  32 query heads of 128 over 8 KV heads: 16,384 tokens of one prompt
// behind 16,384 under a window of 4,096 in 771 us (1.43 PFLOP/s), eight chunks of 2,048
// under one of 1,024 in 253 us (1.09 PFLOP/s, 51 % of the cycles), with fp32 outputs 1,076
// and 348; over E4M3 caches, where two warps widen the codes, 1,224 and 399 us (0.90 and
// 0.69 PFLOP/s, 32 %).
#pragma once

#include "decode_kernel.cuh"
#include "mma_frag.cuh"
#include "tc_utils.cuh"

namespace pkv {

// Element i of a cached row.
template <int KT>
__device__ __forceinline__ float cached(const void* row, int i) {
    if constexpr (KT == kFP8) {
        const uint32_t h = e4m3x2_to_half2(static_cast<const uint8_t*>(row)[i]);
        return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
    } else {
        return Elem<KT>::to_float(static_cast<const typename Elem<KT>::T*>(row)[i]);
    }
}

// One output row on the CUDA cores, by one warp: query head `head` of token `tok`
// (position pos of sequence s); only the keys in sight are read, 32 at a time: a lane
// a key for the scores, then lane l's dims VD*l .. VD*l + VD - 1 of all 32.  What
// makes every element NaN ends it (rows come here by the thousand where a model's
// values are NaN throughout).
template <int DT, int KT, int D>
__device__ __noinline__ void exact_row(const PrefillArgs& a, int s, int h, int64_t tok, int head, int pos) {
    constexpr int VD = D / 32;
    using T = typename Elem<DT>::T;
    const int lane = threadIdx.x & 31;
    const int eb = KT == kFP8 ? 1 : static_cast<int>(sizeof(T));
    const int64_t row = (tok * a.num_q_heads + head) * D;
    const T* q = static_cast<const T*>(a.q) + row;
    const int from = max(0, pos - a.window + 1), first = min(a.sinks, from);
    const int total = first + pos - from + 1;
    float o[VD];
#pragma unroll
    for (int i = 0; i < VD; ++i) o[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int base = 0; base < total; base += 32) {
        const int i = base + lane;
        int64_t r = 0;  // the key's row in the caches
        float x = -INFINITY;
        if (i < total) {
            const int t = i < first ? i : from + i - first;
            int blk = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + t / a.block_size];
            if (blk < 0 || blk >= a.num_blocks) {
                raise_flag(a.status, kFlagBadBlock);
                blk = 0;
            }
            r = (static_cast<int64_t>(blk) * a.num_kv_heads + h) * a.block_size + t % a.block_size;
            const char* k = static_cast<const char*>(a.k_cache) + r * D * eb;
            x = 0.f;
#pragma unroll 8
            for (int d = 0; d < D; ++d) x = fmaf(Elem<DT>::to_float(q[d]) * a.scale_log2, cached<KT>(k, d), x);
        }
        float mn = x;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        mn = fmaxf(m, mn);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float al = fast_exp2(m - ref);
        const float p = i < total ? fast_exp2(x - ref) : 0.f;
        m = mn;
        float sum = p;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = fmaf(l, al, sum);
#pragma unroll
        for (int e = 0; e < VD; ++e) o[e] *= al;
        const int n = min(32, total - base);
        for (int k = 0; k < n; ++k) {
            const float pk = __shfl_sync(0xffffffffu, p, k);
            const int64_t rk = __shfl_sync(0xffffffffu, r, k);
            const char* v = static_cast<const char*>(a.v_cache) + (rk * D + VD * lane) * eb;
#pragma unroll
            for (int e = 0; e < VD; ++e) o[e] = fmaf(pk, cached<KT>(v, e), o[e]);
        }
        bool gone = l != l;
        if (!gone) {
            gone = true;
#pragma unroll
            for (int e = 0; e < VD; ++e) gone = gone && o[e] != o[e];
        }
        if (__all_sync(0xffffffffu, gone)) break;
    }
    const float inv = (KT == kFP8 ? a.v_scale : 1.f) / l;
#pragma unroll
    for (int e = 0; e < VD; ++e) store_out(a.out, row + VD * lane + e, o[e] * inv, a.out_dtype);
}

namespace {

constexpr int kRowsTile = 128;
constexpr int kKeys = 128;
constexpr int kThreads = 384;  // (warps 10 and 11 fill the third warpgroup and do nothing)
// Registers of a thread of the first two warpgroups and of the third: the launch's
// 168 each (65,536 over 384 threads) divided anew, 2 x 208 + 88 = 3 x 168.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr uint32_t kSlice = kRowsTile * 128;  // Q: 128 rows of 64 elements, 16 KiB
constexpr uint32_t kGroup = 8 * 128;          // 8 rows of 64 elements: the swizzle's atom
constexpr uint32_t kTmemCols = 512;
// How far below the maximum a row's reference is set, and the sum of half a tile's
// weights above which it moves.  f16 weights are 2^7 at the maximum then: the largest may
// be 65,504, and below 2^-25 they are lost.  A first token that every query looks at lies
// far above the keys of the window, which may be all that the output is made of where its
// V is near zero: with weights of 1 at the maximum 4,096 keys 2^25.5 below it came out as
// 0 instead of 8.7e-5.  (Another 2^2 leaves too little room before the reference has to
// move: the long chunk took 982 us instead of 841.)  bf16 weights have fp32's exponents.
template <int DT>
__device__ constexpr float kLower = DT == kF16 ? 7.f : 0.f;
template <int DT>
__device__ constexpr float kMoveAt = DT == kF16 ? 65504.f : 4096.f;

template <int D, bool kFP8>
struct Layout {
    static constexpr uint32_t kTile = (D / 64) * kSlice;  // Q of a row tile, K or V of 128 keys
    static constexpr uint32_t kRowGroup = (D / 64) * kGroup;  // K and V: 8 rows of all slices, slice by slice
    // A stage of the ring holds the V of a tile of keys and the K of the next one.
    static constexpr uint32_t kStage = 2 * kTile;
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kRing = 2 * kTile;
    // 4 KiB for each softmax warp: 32 rows of 128 bytes.  An E4M3 cache: the codes of 128 keys' V and K instead.
    static constexpr uint32_t kOut = kRing + kStages * kStage;
    static_assert(!kFP8 || D == 128, "E4M3 rows of 128 codes");
    static constexpr uint32_t kBars = kOut + 8 * 4096;
};

template <int kStages>
struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full[2], q_empty[2];  // of each row tile
    uint64_t s_full[2], o_full[2];
    uint64_t p_full[2];
    uint64_t raw_full[2], raw_empty[2];  // E4M3: the codes of V and of K
    int4 note[8];                       // what each softmax warp needs of its item at the end
    uint32_t tmem;
    int abort;
};

// A place in the ring, going round.
template <int kStages>
struct Place {
    uint32_t stage = 0, round = 0;
    __device__ __forceinline__ Place next() const {
        return stage + 1 == kStages ? Place{0, round + 1} : Place{stage + 1, round};
    }
};

// The rest of a wait that the first look did not end, kept out of the issuing loop.
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
    return mbar_wait_bounded(bar, parity, abort, status);
}

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

// Operand descriptors (see tc_sdesc) from their two words: the high one holds the
// distance of the 8-row groups (and version and swizzle), and a step along an operand
// adds its bytes / 16 to the low one.
__host__ __device__ constexpr uint32_t desc_high(uint32_t group_bytes) { return (group_bytes >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }


// Four MMAs, issued by one elected lane of a converged warp: the whole warp makes the
// descriptors, so they stay in uniform registers and nothing stands between two
// issues (an issue returns about when the MMA before it completes; with the loop in
// a branch of one lane an MMA of 64 cycles took 100).  A and B in shared memory, 32
// bytes (16 elements) a step:
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a_low, uint32_t a_high, uint32_t b_low, uint32_t b_high,
                                        uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred lead, p;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|lead, 0xffffffff;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t"
        "setp.eq.u32 p, 0, 0;\n\t"
        "add.s64 da, da, 2;\n\tadd.s64 db, db, 2;\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t"
        "add.s64 da, da, 2;\n\tadd.s64 db, db, 2;\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t"
        "add.s64 da, da, 2;\n\tadd.s64 db, db, 2;\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(a_high), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A in tensor memory, 8 columns (16 elements) a step; B kStep / 16 further a step.
template <uint32_t kStep>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a_tmem, uint32_t b_low, uint32_t b_high, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred lead, p;\n\t.reg .b64 db;\n\t.reg .b32 ta;\n\t"
        "elect.sync _|lead, 0xffffffff;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 ta, %1;\n\tmov.b64 db, {%2, %3};\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, p;\n\t"
        "setp.eq.u32 p, 0, 0;\n\t"
        "add.s32 ta, ta, 8;\n\tadd.s64 db, db, %6;\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, p;\n\t"
        "add.s32 ta, ta, 8;\n\tadd.s64 db, db, %6;\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, p;\n\t"
        "add.s32 ta, ta, 8;\n\tadd.s64 db, db, %6;\n\t"
        "@lead tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate), "n"(kStep >> 4)
        : "memory");
}

// tc_commit by one elected lane of a converged warp.
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred lead;\n\telect.sync _|lead, 0xffffffff;\n\t"
        "@lead tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
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

__device__ __forceinline__ void tc_ld16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}

// Rows 8 y .. of a cache, all 64-element slices (the map's third axis).
__device__ __forceinline__ void tensor_load_4d(void* dst, const CUtensorMap* map, int y, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %2, %2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(smem_addr(bar)), "l"(policy)
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

// 64 columns of tensor memory; what reads them stays behind the wait for them (hold64).
__device__ __forceinline__ void load64(uint32_t col, float (&s)[64]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float x[32];
        tc_ld32(col + 32 * q, x);
#pragma unroll
        for (int c = 0; c < 32; ++c) s[32 * q + c] = x[c];
    }
}
__device__ __forceinline__ void hold64(float (&s)[64]) {
#pragma unroll
    for (int c = 0; c < 64; c += 16)
        asm volatile("" : "+f"(s[c]), "+f"(s[c + 1]), "+f"(s[c + 2]), "+f"(s[c + 3]), "+f"(s[c + 4]), "+f"(s[c + 5]),
                          "+f"(s[c + 6]), "+f"(s[c + 7]), "+f"(s[c + 8]), "+f"(s[c + 9]), "+f"(s[c + 10]), "+f"(s[c + 11]),
                          "+f"(s[c + 12]), "+f"(s[c + 13]), "+f"(s[c + 14]), "+f"(s[c + 15]));
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

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (DT == kBF16) {
        const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&w);
        return make_float2(__low2float(h), __high2float(h));
    } else {
        const __half2 h = *reinterpret_cast<const __half2*>(&w);
        return make_float2(__low2float(h), __high2float(h));
    }
}

// Two E4M3 codes (bytes kPair and kPair + 1 of a word) as two values of DT, exactly, in
// integer operations: a code's seven magnitude bits are the low exponent bits and the
// first fraction bits of an f16 or bf16, at 2^-8 or 2^-120 times its value (subnormals
// too).  f16 values stay so (code_scale makes up for it); bf16 ones, whose products
// would leave fp32's range, are multiplied back.
template <int DT, int kPair>
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
    const uint32_t t = __byte_perm(codes, 0u, kPair == 0 ? 0x1404u : 0x3424u);  // in the high bytes of the halves
    if constexpr (DT == kF16) return e4m3x2_odd_bytes_to_half2_shifted(t);
    const uint32_t b = ((t >> 4) & 0x07F007F0u) | (t & 0x80008000u);
    const __nv_bfloat162 up = __float2bfloat162_rn(0x1p120f);
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), up);
    return *reinterpret_cast<const uint32_t*>(&x);
}
template <int DT, bool kFP8>
__host__ __device__ constexpr float code_scale() {
    return kFP8 && DT == kF16 ? 256.f : 1.f;
}

// The rows from w0 on, 32 at most, of each of the CTA's items, as the calling warp wrote them: where they are NaN, again.
// (Out of the kernel's text: there it took registers from the softmax, eight chunks 267 us instead of 253.)
template <int DT, int KT, int D, int G, bool kTwo>
__device__ __noinline__ void nan_rows_again(const PrefillArgs& a, int64_t items, int tiles, int w0) {
    const int lane = threadIdx.x & 31;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int h = static_cast<int>(i / tiles);
        const int4 u = __ldcg(reinterpret_cast<const int4*>(a.tiles) + 2 * (i - static_cast<int64_t>(h) * tiles));
        for (int row = w0; row < min(w0 + 32, u.z * G); ++row) {  // (u: sequence, first token, tokens, position)
            const int64_t tok = u.y + row / G, o0 = (tok * a.num_q_heads + h * G + row % G) * D;
            bool nan = false;
            for (int d = lane; d < D; d += 32) {
                float o;
                if constexpr (kTwo)
                    o = static_cast<const float*>(a.out)[o0 + d];
                else
                    o = Elem<DT>::to_float(static_cast<const typename Elem<DT>::T*>(a.out)[o0 + d]);
                nan = nan || o != o;
            }
            if (__any_sync(0xffffffffu, nan)) exact_row<DT, KT, D>(a, u.x, h, tok, h * G + row % G, u.w + row / G);
        }
    }
}

// kTwo: P in two parts.  kFP8: an E4M3 cache; its codes come by bulk copies, and warps
// 10 and 11 widen them to q's type in the stages, exactly.
template <int DT, int D, int G, bool kTwo, bool kFP8>
__global__ void __launch_bounds__(kThreads, 1) paged_window_prefill_tc_kernel(const PrefillArgs a,
                                                                               const __grid_constant__ CUtensorMap tmq,
                                                                               const __grid_constant__ CUtensorMap tmk,
                                                                               const __grid_constant__ CUtensorMap tmv) {
    using L = Layout<D, kFP8>;
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
            mbar_init(&B->full[i], kFP8 ? 2 : 1);  // the widening warps, or the copies' bytes
            mbar_init(&B->empty[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&B->q_full[t], 1);
            mbar_init(&B->q_empty[t], 1);
            mbar_init(&B->s_full[t], 1);
            mbar_init(&B->p_full[t], 4);
            mbar_init(&B->o_full[t], 1);
            mbar_init(&B->raw_full[t], 1);
            mbar_init(&B->raw_empty[t], 2);
        }
        B->abort = 0;
        fence_barrier_init();
        prefetch_tensor_map(&tmq);
        if constexpr (!kFP8) {
            prefetch_tensor_map(&tmk);
            prefetch_tensor_map(&tmv);
        }
    }
    if (warp == 9) tc_alloc(&B->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = B->tmem;
    pdl_wait();

    const int tiles = a.tile_cum[a.num_seqs];
    const int64_t items = static_cast<int64_t>(tiles) * a.num_kv_heads;
    const int sh = a.box == 32 ? 5 : 4, box = 1 << sh;
    const int per_tile = kKeys >> sh;  // boxes of a tile
    auto item_at = [&](int64_t i) {
        Item it;
        it.h = static_cast<int>(i / tiles);
        const int4* d = reinterpret_cast<const int4*>(a.tiles) + 2 * (i - static_cast<int64_t>(it.h) * tiles);
        const int4 u = __ldcg(d), v = __ldcg(d + 1);
        it.s = u.x;
        it.tok0 = u.y;
        it.ntok = u.z;
        it.pos0 = u.w;
        it.ctx = v.x;
        const int lo = max(0, it.pos0 - a.window + 1) >> sh, sb = static_cast<int>((static_cast<int64_t>(a.sinks) + box - 1) >> sh);
        const int skip = max(0, lo - sb);
        it.skip = skip << sh;
        it.sink_keys = static_cast<int>(min(static_cast<int64_t>(sb) << sh, int64_t{0x7fffffff}));
        it.boxes = ((it.pos0 + it.ntok - 1) >> sh) + 1 - skip;
        it.tiles = (it.boxes + per_tile - 1) >> (7 - sh);
        return it;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity & 1u, abort, a.status); };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            // ---- producer
            const uint64_t keep = policy_evict_last();
            Place<kStages> at;
            uint32_t nq[2] = {0, 0}, nraw[2] = {0, 0};
            bool ok = true;
            // The cache's 8-row group of box `lane` of tile j (the same for K and V); a box lies within a block.
            auto group_of = [&](const Item& it, int j) {
                if (lane >= per_tile || j >= it.tiles) return 0;
                const int b = j * per_tile + lane;
                const int cg = b < it.boxes ? b << sh : 0;  // (behind the last box: the first again, masked)
                const int key = cg + (cg >= it.sink_keys ? it.skip : 0);
                const int lb = key / a.block_size;
                int blk = a.block_tables[static_cast<int64_t>(it.s) * a.max_blocks + lb];
                if (blk < 0 || blk >= a.num_blocks) {
                    raise_flag(a.status, kFlagBadBlock);
                    blk = 0;
                }
                return ((blk * a.num_kv_heads + it.h) * a.block_size + (key - lb * a.block_size)) >> 3;
            };
            // A stage: the V of a tile (groups yv, a box a lane; first time round: none) and the K of the next (yk).
            auto load = [&](bool v, int yv, bool k, int yk) -> bool {
                int good = 1;
                if constexpr (kFP8) {  // into the room for codes, as soon as it has been widened
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        if (p == 0 ? !v : !k) continue;
                        if (lane == 0) {
                            if (nraw[p] > 0) good = wait(&B->raw_empty[p], nraw[p] - 1);
                            if (good) mbar_arrive_expect_tx(&B->raw_full[p], kKeys * D);
                        }
                        good = __shfl_sync(0xffffffffu, good, 0);
                        if (!good) return false;
                        ++nraw[p];
                        if (lane < per_tile)
                            bulk_load(base + L::kOut + p * kKeys * D + lane * box * D,
                                      static_cast<const char*>(p == 0 ? a.v_cache : a.k_cache) +
                                          static_cast<int64_t>(p == 0 ? yv : yk) * (8 * D),
                                      box * D, &B->raw_full[p], keep);
                        __syncwarp();
                    }
                    return true;
                }
                if (lane == 0) {
                    if (at.round > 0) good = wait(&B->empty[at.stage], at.round - 1);
                    if (good) mbar_arrive_expect_tx(&B->full[at.stage], (v ? L::kTile : 0u) + (k ? L::kTile : 0u));
                }
                good = __shfl_sync(0xffffffffu, good, 0);
                if (!good) return false;
                if (lane < per_tile) {
                    uint8_t* dst = base + L::kRing + at.stage * L::kStage + lane * (box / 8) * L::kRowGroup;
                    if (v) tensor_load_4d(dst, &tmv, yv, &B->full[at.stage], keep);
                    if (k) tensor_load_4d(dst + L::kTile, &tmk, yk, &B->full[at.stage], keep);
                }
                __syncwarp();
                at = at.next();
                return true;
            };
            // The row tiles of an item's Q, each once the S of the item before are done with its buffer.
            auto load_q = [&](const Item& it) -> bool {
                int good = 1;
                if (lane == 0) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t * kTileTokens >= it.ntok || !good) continue;
                        if (nq[t] > 0) good = wait(&B->q_empty[t], nq[t] - 1);
                        if (!good) continue;
                        mbar_arrive_expect_tx(&B->q_full[t], L::kTile);
                        for (int sl = 0; sl < kSlices; ++sl)
                            tensor_load_3d(base + L::kQ + t * L::kTile + sl * kSlice, &tmq, sl * 64, it.h * G,
                                           static_cast<int>(it.tok0) + t * kTileTokens, &B->q_full[t], keep);
                        ++nq[t];
                    }
                }
                return __shfl_sync(0xffffffffu, good, 0) != 0;
            };
            Item it;
            int y = 0;
            if (blockIdx.x < items) {
                it = item_at(blockIdx.x);
                y = group_of(it, 0);
                ok = load(false, 0, true, y) && load_q(it);
            }
            for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
                const bool more = i + gridDim.x < items;
                Item next = it;
                if (more) next = item_at(i + gridDim.x);
                for (int j = 0; j < it.tiles && ok; ++j) {
                    const bool ends = j + 1 == it.tiles;
                    const int y_next = !ends ? group_of(it, j + 1) : more ? group_of(next, 0) : 0;
                    ok = load(true, y, !ends || more, y_next);
                    y = y_next;
                }
                if (ok && more) ok = load_q(next);
                it = next;
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
                    const uint32_t fills = at.round + (st < at.stage ? 1u : 0u);
                    if (fills > 0) drain(&B->full[st], fills - 1);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (nq[t] > 0) drain(&B->q_full[t], nq[t] - 1);
                    if (kFP8 && nraw[t] > 0) drain(&B->raw_full[t], nraw[t] - 1);
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---- MMA issue: the warp as one, an elected lane where an instruction is one thread's
            constexpr int bf = DT == kBF16 ? 1 : 0;
            constexpr uint32_t idS = tc_idesc_f16(bf, false, kKeys, kRowsTile);
            constexpr uint32_t idPV = tc_idesc_f16(bf, true, D, kRowsTile);
            const uint32_t qa = smem_addr(base + L::kQ), ring = smem_addr(base + L::kRing);
            uint32_t nq = 0, np = 0;  // phases of Q's and P's barriers, row tile 1's in the upper halves
            auto count = [](uint32_t& n, int t) {
                const uint32_t x = n >> (16 * t);
                n = t ? n + 0x10000u : (n & 0xffff0000u) | ((n + 1) & 0xffffu);
                return x;
            };
            using At = Place<kStages>;
            At at;  // stage of a step's V and of the next step's K
            // (A wait is as few instructions as it can be: the softmax warps of this sub-partition issue in between.)
            auto done = [&](uint64_t* bar, uint32_t parity) {
                while (!mbar_try_wait(bar, parity & 1u))
                    if (!wait_longer(bar, parity & 1u, abort, a.status)) break;  // (the flag is set: see the end of a step)
                __syncwarp();
            };
            auto qk = [&](int t, const At& x) {
                const uint32_t k = desc_low(ring + x.stage * L::kStage + L::kTile, 16), q = desc_low(qa + t * L::kTile, 16);
#pragma unroll
                for (int sl = 0; sl < kSlices; ++sl)
                    mma4_ss(taddr + t * kKeys, q + (sl * kSlice >> 4), desc_high(kGroup), k + (sl * kGroup >> 4),
                            desc_high(L::kRowGroup), idS, sl > 0);
                commit_elected(&B->s_full[t]);
            };
            auto pv = [&](int t, const At& x, bool first) {
                const uint32_t va = desc_low(ring + x.stage * L::kStage, kGroup);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)  // half the keys
#pragma unroll
                    for (int part = 0; part < (kTwo ? 2 : 1); ++part)
                        mma4_ts<2 * L::kRowGroup>(taddr + 256 + t * 128, taddr + t * kKeys + hf * 64 + part * 32,
                                                  va + (hf * 8 * L::kRowGroup >> 4), desc_high(L::kRowGroup), idPV,
                                                  !(first && part == 0 && hf == 0));
            };
            // S of the row tiles of a step (a tile of an item's keys), K at ring position x; `fresh`: the
            // item's first, `left` 1: its last.
            struct Step {
                int row_tiles, left;  // tiles of the item from this one on
                bool fresh;
            };
            auto qk_of = [&](int t, const At& x, const Step& n) {
                qk(t, x);
                if (n.left == 1) commit_elected(&B->q_empty[t]);
            };
            int64_t i = blockIdx.x;
            auto first_step = [&](int64_t x) {
                if (x >= items) return Step{0, 0, true};
                const Item it = item_at(x);
                return Step{it.ntok > kTileTokens ? 2 : 1, it.tiles, true};
            };
            Step now = first_step(i), item_next = first_step(i + gridDim.x);
            if (now.row_tiles > 0) {
                done(&B->full[at.stage], at.round);
#pragma unroll 1
                for (int t = 0; t < now.row_tiles; ++t) {
                    done(&B->q_full[t], count(nq, t));
                    tc_fence_after();
                    qk_of(t, at, now);
                }
                commit_elected(&B->empty[at.stage]);
                at = at.next();
            }
            while (now.row_tiles > 0 && !*abort) {
                // P . V of this step, and S of the next one, row tile by row tile: an item's first S stand between
                // the last P . V of the item before, while its rows are written out.  Waits come before the first
                // issue: an issue returns when the MMA before it is done, so that the tensor cores stand still
                // while this warp looks at a barrier.
                const bool ends = now.left == 1;
                const Step next = ends ? item_next : Step{now.row_tiles, now.left - 1, false};
                done(&B->full[at.stage], at.round);
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const bool more = t < next.row_tiles;
                    if (more && next.fresh) done(&B->q_full[t], count(nq, t));
                    if (t < now.row_tiles) {
                        done(&B->p_full[t], count(np, t));
                        tc_fence_after();
                        pv(t, at, now.fresh);
                        if (ends) commit_elected(&B->o_full[t]);
                    } else {
                        tc_fence_after();
                    }
                    if (more) qk_of(t, at, next);
                }
                commit_elected(&B->empty[at.stage]);
                at = at.next();
                now = next;
                if (ends) {
                    i += gridDim.x;
                    item_next = first_step(i + gridDim.x);
                }
            }
            __syncwarp();
        } else if constexpr (kFP8) {
            // ---- warps 10 and 11: the codes of 64 keys each, stage by stage, V before K
            Place<kStages> at;
            uint32_t n[2] = {0, 0};
            const int row0 = (warp - 10) * 64;
            uint32_t to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t r = (lane >> 4) + 2 * u, q = lane & 15;
                to[u] = (q >> 3) * kGroup + r * 128 + (((q & 7) ^ r) << 4);
            }
            auto widen = [&](bool v, bool k) -> bool {
                if (at.round > 0 && !__all_sync(0xffffffffu, wait(&B->empty[at.stage], at.round - 1))) return false;
                uint8_t* stage = base + L::kRing + at.stage * L::kStage;
#pragma unroll 1
                for (int p = 0; p < 2; ++p) {
                    if (p == 0 ? !v : !k) continue;
                    const uint32_t nth = p == 0 ? n[0]++ : n[1]++;
                    if (!__all_sync(0xffffffffu, wait(&B->raw_full[p], nth))) return false;
                    const uint8_t* raw = base + L::kOut + p * kKeys * D;
                    const uint8_t* src = raw + (row0 + (lane >> 4)) * D + (lane & 15) * 8;
                    uint8_t* dst = stage + p * L::kTile + (row0 >> 3) * L::kRowGroup;
                    // 8 rows at a time, two by two: lane / 16 + 2 u is the row, lane % 16 its chunk of 8 codes.
#pragma unroll 2
                    for (int g = 0; g < 8; ++g) {
                        uint2 c[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) c[u] = *reinterpret_cast<const uint2*>(src + (8 * g + 2 * u) * D);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            *reinterpret_cast<uint4*>(dst + g * L::kRowGroup + to[u]) =
                                make_uint4(widen2<DT, 0>(c[u].x), widen2<DT, 2>(c[u].x), widen2<DT, 0>(c[u].y),
                                           widen2<DT, 2>(c[u].y));
                    }
                    fence_proxy_async_smem();  // before the tensor cores read it (and before the next codes come)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B->raw_empty[p]);
                }
                if (lane == 0) mbar_arrive(&B->full[at.stage]);
                at = at.next();
                return true;
            };
            bool ok = blockIdx.x >= items || widen(false, true);
            for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
                const int tiles = item_at(i).tiles;
                for (int j = 0; j < tiles && ok; ++j) ok = widen(true, j + 1 < tiles || i + gridDim.x < items);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---- softmax: thread r of warps 4t .. 4t + 3 owns row r of row tile t
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lane_base = taddr + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t s_col = lane_base + t * kKeys, o_col = lane_base + 256 + t * 128;
        const float sc = fmaxf(fabsf(a.scale_log2) * code_scale<DT, kFP8>(), 1e-30f);  // (zero: every finite score's exponent is 0)
        const bool negative = a.scale_log2 < 0.f;
        uint32_t ns = 0, no = 0, at = 0;
        bool ok = true;
        bool again = false;  // this warp wrote a row that is NaN
        Item it;
        if (blockIdx.x < items) it = item_at(blockIdx.x);
        for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
            if (t * kTileTokens >= it.ntok) {  // (row tile 1 of a short item)
                at += it.tiles;
                if (i + gridDim.x < items) it = item_at(i + gridDim.x);
                continue;
            }
            const int num_tiles = it.tiles;
            // Keys in sight of the row, as places in the list: [0, va) and [vb, vc).  All rows of the warp (32 / G
            // tokens) see all keys of the halves of tiles [whole_from, whole_to); with a negative scale, whose sign
            // the masking applies, there are none.
            int va, vb, vc, whole_from, whole_to;
            {
                const int w0 = t * kTileTokens + (warp & 3) * 32 / G, tr = t * kTileTokens + r / G;
                const int p = it.pos0 + min(tr, it.ntok - 1);
                const int p0 = it.pos0 + min(w0, it.ntok - 1), p1 = it.pos0 + min(w0 + 31 / G, it.ntok - 1);
                va = min(a.sinks, p + 1);
                vb = max(0, p - a.window + 1 - it.skip);
                vc = p + 1 - it.skip;
                whole_from = (max(0, p1 - a.window + 1 - it.skip) + 63) >> 6;
                whole_to = negative ? 0 : (p0 + 1 - it.skip) >> 6;
            }
            if (lane == 0) B->note[warp] = make_int4(it.h, it.ntok, static_cast<int>(it.tok0), 0);
            const int live = it.ctx - it.skip;  // places from there on hold no token
            float m_ref = -INFINITY, l = 0.f;
            float limit = -1.f;  // of a half tile's sum of weights: kMoveAt once there is a reference
            // Half a tile's keys: mask, weights, P.
            auto half = [&](float (&sv)[64], int j, int hf) -> bool {
                if (2 * j + hf < whole_from || 2 * j + hf >= whole_to) {  // (else every row of the warp sees all 64)
                    const int k0 = j * kKeys + hf * 64;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int c0 = k0 + 32 * q;
                        const uint32_t seen = columns(0, va - c0) | columns(vb - c0, vc - c0);
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float x = negative ? -sv[32 * q + c] : sv[32 * q + c];
                            sv[32 * q + c] = (seen >> c) & 1u ? x : -INFINITY;
                        }
                    }
                }
                uint32_t hi[32];
                [[maybe_unused]] uint32_t lo[kTwo ? 32 : 1];
                float sum = 0.f;
                auto weights = [&]() {
                    const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
                    const float2 sc2 = make_float2(sc, sc), neg2 = make_float2(neg, neg);
                    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float2 e = fma2(make_float2(sv[2 * c], sv[2 * c + 1]), sc2, neg2);
                        const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                        part[c & 1] = add2(part[c & 1], p);
                        if constexpr (kTwo)
                            pack_split<DT>(p.x, p.y, hi[c], lo[c]);
                        else
                            hi[c] = pack2<DT>(p.x, p.y);
                    }
                    const float2 both = add2(part[0], part[1]);
                    sum = both.x + both.y;
                };
                auto store = [&]() {  // over the S that they came from
                    tc_st32u(s_col + 64 * hf, hi);
                    if constexpr (kTwo) tc_st32u(s_col + 64 * hf + 32, lo);
                };
                weights();
                store();  // (before it is known whether they stand, so that the vote costs nothing)
                if (__any_sync(0xffffffffu, !(sum <= limit))) {
                    tc_wait_st();
                    // A new reference by the maximum of these scores.  (S being there says that the P . V before are
                    // done.)
                    float mx = sv[0];
#pragma unroll
                    for (int c = 1; c < 64; ++c) mx = fmaxf(mx, sv[c]);
                    mx = mx * sc - kLower<DT>;
                    const bool move = mx > m_ref && !(sum <= limit);
                    // The step is a whole number, so that it scales what stands in P exactly (down to f16's last place);
                    // it is 2 at least, or the sum would not have passed the limit.
                    if (m_ref > -INFINITY) mx = m_ref + floorf(mx - m_ref);
                    const float f = move ? fast_exp2(m_ref - mx) : 1.f;  // (0 from -inf)
                    if (move) {
                        l *= f;
                        m_ref = mx;
                        limit = kMoveAt<DT>;
                    }
                    if (j > 0) {
#pragma unroll
                        for (int cb = 0; cb < D / 16; ++cb) {
                            float o[16];
                            tc_ld16(o_col + 16 * cb, o);
                            tc_wait_ld();
                            uint32_t u[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(o[c] * f);
                            tc_st16u(o_col + 16 * cb, u);
                        }
                    }
                    if (hf == 1) {  // the first half's weights
#pragma unroll
                        for (int cb = 0; cb < (kTwo ? 4 : 2); ++cb) {
                            float w[16];
                            tc_ld16(s_col + 16 * cb, w);
                            tc_wait_ld();
                            uint32_t u[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const float2 x = unpack2<DT>(__float_as_uint(w[c]));
                                u[c] = pack2<DT>(x.x * f, x.y * f);
                            }
                            tc_st16u(s_col + 16 * cb, u);
                        }
                    }
                    weights();
                    store();
                }
                l += sum;
                if (hf == 0 && t == 0 && (j + 1) * kKeys > live) {
                    const uint32_t st = (at + 1) % kStages;  // (stage 0 of round 0 holds the first K alone)
                    if (!__all_sync(0xffffffffu, wait(&B->full[st], (at + 1) / kStages))) return false;
                    const int from = max(0, live - j * kKeys);
                    uint8_t* vd = base + L::kRing + st * L::kStage;
                    for (int e = r; e < (kKeys - from) * 8 * kSlices; e += 128) {
                        const int row = from + e / (8 * kSlices), c = e % (8 * kSlices);
                        *reinterpret_cast<uint4*>(vd + (row >> 3) * L::kRowGroup + (c >> 3) * kGroup + (row & 7) * 128 +
                                                  ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                return true;
            };
            auto give = [&]() {  // P to the issuing warp
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_full[t]);
                ++at;
            };
            // With a P of one part the second half's S is on its way while the first is worked on (long chunk 819 ->
            // 783 us); a P of two parts and the E4M3 kernel's roles, which need the registers and the instruction
            // cache, take one text for both halves (two-part chunks 369 us, 413 with the other).
            if constexpr (!kTwo && !kFP8) {
#pragma unroll 1
                for (int j = 0; j < num_tiles && ok; ++j) {
                    ok = __all_sync(0xffffffffu, wait(&B->s_full[t], ns++));
                    if (!ok) break;
                    tc_fence_after();
                    float s0[64], s1[64];
                    load64(s_col, s0);
                    tc_wait_ld();
                    hold64(s0);
                    load64(s_col + 64, s1);
                    ok = half(s0, j, 0);
                    tc_wait_ld();
                    hold64(s1);
                    if (!ok) break;
                    half(s1, j, 1);
                    give();
                }
            } else {
#pragma unroll 1
                for (int hh = 0; hh < 2 * num_tiles && ok; ++hh) {
                    const int j = hh >> 1, hf = hh & 1;
                    if (hf == 0) {
                        ok = __all_sync(0xffffffffu, wait(&B->s_full[t], ns++));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    float sv[64];
                    load64(s_col + 64 * hf, sv);
                    tc_wait_ld();
                    hold64(sv);
                    ok = half(sv, j, hf);
                    if (hf == 1) give();
                }
            }
            if (!ok) break;
            __syncwarp();
            const int4 note = B->note[warp];  // (not held through the loop above: its registers are all in use)
            const int64_t tok0 = note.z;
            if (i + gridDim.x < items) it = item_at(i + gridDim.x);
            ok = __all_sync(0xffffffffu, wait(&B->o_full[t], no++));
            if (!ok) break;
            tc_fence_after();
            const int w0 = t * kRowsTile + (warp & 3) * 32;  // the warp's first row of the item
            const int rows = min(32, note.y * G - w0);       // its rows that are the item's
            const float inv = (kFP8 ? a.v_scale * code_scale<DT, kFP8>() : 1.f) / l;
            bool nan = false;
            // 32 rows of 128 bytes at a time through shared memory, so that a store takes whole rows' pieces (an E4M3
            // cache's codes take that room: each thread stores its own row).
            [[maybe_unused]] uint8_t* stage = base + L::kOut + warp * 4096;
            constexpr int kPer = kTwo ? 32 : 64;  // elements of 128 bytes
#pragma unroll
            for (int cb = 0; cb < D / kPer; ++cb) {
                uint32_t w[32];
#pragma unroll
                for (int q = 0; q < kPer / 32; ++q) {
                    float o[32];
                    tc_ld32(o_col + kPer * cb + 32 * q, o);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        o[c] *= inv;
                        nan = nan || o[c] != o[c];
                    }
                    if constexpr (kTwo) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) w[c] = __float_as_uint(o[c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c) w[16 * q + c] = pack2<DT>(o[2 * c], o[2 * c + 1]);
                    }
                }
                if (cb == D / kPer - 1) tc_fence_before();  // O is read before this thread lets the next P . V begin
                if constexpr (kFP8) {
                    if (lane < rows) {
                        const int64_t o0 = ((tok0 + (w0 + lane) / G) * a.num_q_heads + note.x * G + (w0 + lane) % G) * D;
                        char* dst = static_cast<char*>(a.out) + (o0 + kPer * cb) * (kTwo ? 4 : 2);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    }
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int row = 4 * q + (lane >> 3), c = lane & 7;
                    if (row < rows) {
                        const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 128 + ((c ^ (row & 7)) << 4));
                        const int64_t o0 = ((tok0 + (w0 + row) / G) * a.num_q_heads + note.x * G + (w0 + row) % G) * D;
                        *reinterpret_cast<uint4*>(static_cast<char*>(a.out) + (o0 + kPer * cb) * (kTwo ? 4 : 2) + 16 * c) = x;
                    }
                }
                __syncwarp();
            }
            again = again || (nan && lane < rows);
        }
        // The rows that this warp wrote as NaN, again (see above).
        __syncwarp();
        if (ok && __any_sync(0xffffffffu, again))
            nan_rows_again<DT, kFP8 ? static_cast<int>(pkv::kFP8) : DT, D, G, kTwo>(a, items, tiles,
                                                                                   t * kRowsTile + (warp & 3) * 32);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tc_dealloc(taddr, kTmemCols);
    }
}

template <int DT, int D, int G, bool kTwo, bool kFP8>
cudaError_t launch_tc(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int ctas,
                      cudaStream_t stream) {
    static RaisedLimit limit;
    auto kern = paged_window_prefill_tc_kernel<DT, D, G, kTwo, kFP8>;
    const cudaError_t e = allow_shared_memory(kern, a.device, a.smem_bytes, &limit);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(ctas), dim3(kThreads), static_cast<size_t>(a.smem_bytes), stream, a.pdl != 0, a, tmq, tmk,
                         tmv);
}

template <int DT, int D, bool kTwo, bool kFP8 = false>
cudaError_t launch_tc_g(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int ctas,
                        cudaStream_t stream) {
    switch (a.num_q_heads / a.num_kv_heads) {
        case 1: return launch_tc<DT, D, 1, kTwo, kFP8>(a, tmq, tmk, tmv, ctas, stream);
        case 2: return launch_tc<DT, D, 2, kTwo, kFP8>(a, tmq, tmk, tmv, ctas, stream);
        case 4: return launch_tc<DT, D, 4, kTwo, kFP8>(a, tmq, tmk, tmv, ctas, stream);
        case 8: return launch_tc<DT, D, 8, kTwo, kFP8>(a, tmq, tmk, tmv, ctas, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace pkv
