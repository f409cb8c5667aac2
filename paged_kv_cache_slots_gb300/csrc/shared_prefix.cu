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
// left to the split-context decode kernel.  Three launches:
//   parts   (this file's main kernel) (m, l, O) of 128 rows over a chunk of a
//           group's keys, one CTA a (group, KV head, row tile, chunk);
//   tails   the decode kernel over the tokens after the prefix, partials only;
//   merge   one warp a (sequence, query head).
// parts and tails are independent and run side by side as far as there is
// room.  Which sequences share (those at least as long as the prefix; shorter
// ones read their own tables throughout) and how the keys are cut follows from
// the groups alone, so every CTA works it out for itself: one warp-wide pass
// over the groups costs less than a launch that does it for all.
//
// The parts kernel is built like the prefill kernel (prefill_tc.cu): a
// producer brings K and V tiles of 64 keys into swizzled shared memory, one
// lane issues tcgen05 MMAs S = Q K^T (tensor memory, two buffers) and
// O += P V (P read from tensor memory), four warps hold the softmax, one row a
// thread.  P enters the product as a high and a low half-precision part, so
// that the result carries fp32-like weights whatever the output type.
#include "decode_kernel.cuh"
#include "mma_frag.cuh"
#include "shared_prefix.cuh"
#include "tc_utils.cuh"

namespace pkv {

namespace {

// ------------------------------------------------------------------ units

constexpr int kMinChunk = 4;  // key tiles a CTA

// The prefix part's work is key tiles: every (group, KV head, row tile) triple
// has the group's tiles, triples in that order.  CTA c of P takes tiles
// [c W / P, (c + 1) W / P), whatever triples they belong to: all CTAs have the
// same work to within a tile.  A run of one triple's tiles in one CTA is a
// segment, and leaves one part.  Part k of a triple comes from the k-th CTA
// that has tiles of it; a group reserves keys P / W + 2 parts of each of its
// rows, so all groups together reserve at most 128 P + 2 (all rows).

// a * b / c for 0 <= a, b and c > 0.
__device__ __forceinline__ int mul_div(int a, int b, int c) {
    const uint64_t p = static_cast<uint64_t>(static_cast<uint32_t>(a)) * static_cast<uint32_t>(b);
    if ((p >> 32) == 0) return static_cast<int>(static_cast<uint32_t>(p) / static_cast<uint32_t>(c));
    return static_cast<int>(p / static_cast<uint32_t>(c));
}

// CTA that owns tile x of W.
__device__ __forceinline__ int cta_of_tile(int x, int W, int P) {
    const uint64_t p = (static_cast<uint64_t>(x) + 1) * static_cast<uint32_t>(P) - 1;
    if ((p >> 32) == 0) return static_cast<int>(static_cast<uint32_t>(p) / static_cast<uint32_t>(W));
    return static_cast<int>(p / static_cast<uint32_t>(W));
}

// One lane's group.
struct GroupShape {
    int seq0, rows, tiles, keys, blocks;  // rows: sequences x G; tiles: row tiles; keys: key tiles
};

__device__ __forceinline__ int group_work(const GroupShape& p, int Hkv) { return Hkv * p.tiles * p.keys; }

// Group g's shape; no work for one past the last.  *bad: it is out of order.
__device__ __forceinline__ GroupShape group_shape(const SharedPrefixArgs& a, int g, int G, bool* bad) {
    GroupShape p{0, 0, 0, 0, 0};
    if (g >= a.num_groups) return p;
    const int s0 = a.group_start[g], s1 = a.group_start[g + 1], len = a.prefix_lens[g];
    if (s0 < 0 || s1 > a.num_seqs || s0 > s1 || len < 0) {
        *bad = true;
        return p;
    }
    p.seq0 = s0;
    p.rows = (s1 - s0) * G;
    p.tiles = (p.rows + 127) >> 7;
    p.blocks = len / a.block_size;
    if (p.blocks > a.max_blocks) p.blocks = 0;  // no sequence is that long
    p.keys = (p.blocks * a.block_size + kPrefixTile - 1) / kPrefixTile;
    return p;
}

// What every CTA, and every warp of it, works out alike.
struct Units {
    GroupShape first;  // this lane's group of the first 32
    int W, P;          // tiles and CTAs with work; W = 0: nothing is shared
};

__device__ __forceinline__ Units plan_units(const SharedPrefixArgs& a, int G) {
    const int lane = threadIdx.x & 31;
    Units u;
    bool bad = false;
    u.first = group_shape(a, lane, G, &bad);
    int work = group_work(u.first, a.num_kv_heads), triples = u.first.keys ? u.first.tiles : 0;
    for (int g0 = 32; g0 < a.num_groups; g0 += 32) {
        const GroupShape p = group_shape(a, g0 + lane, G, &bad);
        work += group_work(p, a.num_kv_heads);
        triples += p.keys ? p.tiles : 0;
    }
    bad = __any_sync(0xffffffffu, bad);
    work = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(work)));
    triples = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(triples))) * a.num_kv_heads;
    u.W = bad ? 0 : work;
    // With little work a CTA has an SM to itself, and four tiles (below that
    // its start and the merge of its parts cost more than its tiles); with
    // more, two share an SM.
    const int all = a.num_sms * a.ctas_per_sm;
    int P = u.W / kMinChunk >= all ? all : min(a.num_sms, (u.W + kMinChunk - 1) / kMinChunk);
    // CTAs that begin with a triple have one segment: worth up to a quarter of
    // the CTAs while a CTA has few tiles, a sixteenth always.
    if (triples > 0 && triples <= P) {
        const int even = P / triples * triples;
        if ((P - even) * (u.W / P < 16 ? 4 : 16) <= P) P = even;
    }
    u.P = P > 0 ? P : 1;
    return u;
}

// A triple, and a tile in it.
struct Triple {
    int seq0, rows, blocks, keys;
    int h, rt;       // KV head, row tile
    int tile0;       // first tile of the triple
    int row0;        // row tile's first partial row, part 0
    int stride;      // rows from one part to the next
};

// The triple of tile x, by the whole warp (0 <= x < W).
__device__ __forceinline__ Triple find_triple(const SharedPrefixArgs& a, const Units& u, int G, int x) {
    const int lane = threadIdx.x & 31;
    Triple t{};
    int tile0 = 0, row0 = 0;
    bool bad = false;
    for (int g0 = 0; g0 < a.num_groups; g0 += 32) {
        const GroupShape p = g0 == 0 ? u.first : group_shape(a, g0 + lane, G, &bad);
        const int work = group_work(p, a.num_kv_heads);
        const int parts = mul_div(p.keys, u.P, u.W) + 2;
        const int rows = p.keys ? a.num_kv_heads * parts * p.rows : 0;
        int w = work, r = rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int yw = __shfl_up_sync(0xffffffffu, w, o), yr = __shfl_up_sync(0xffffffffu, r, o);
            if (lane >= o) w += yw, r += yr;
        }
        const uint32_t mine = __ballot_sync(0xffffffffu, x < tile0 + w);
        if (mine) {
            const int src = __ffs(mine) - 1;
            t.seq0 = __shfl_sync(0xffffffffu, p.seq0, src);
            t.rows = __shfl_sync(0xffffffffu, p.rows, src);
            t.blocks = __shfl_sync(0xffffffffu, p.blocks, src);
            t.keys = __shfl_sync(0xffffffffu, p.keys, src);
            const int tiles = __shfl_sync(0xffffffffu, p.tiles, src);
            const int np = __shfl_sync(0xffffffffu, parts, src);
            const int first = tile0 + __shfl_sync(0xffffffffu, w - work, src);
            const int k = (x - first) / t.keys;
            t.h = k / tiles;
            t.rt = k - t.h * tiles;
            t.tile0 = first + k * t.keys;
            t.stride = t.rows;
            t.row0 = row0 + __shfl_sync(0xffffffffu, r - rows, src) + t.h * np * t.rows + t.rt * 128;
            return t;
        }
        tile0 += __shfl_sync(0xffffffffu, w, 31);
        row0 += __shfl_sync(0xffffffffu, r, 31);
    }
    return t;
}

// Tells the merge where every (sequence, KV head)'s parts are.  One warp.
__device__ void write_parts_table(const SharedPrefixArgs& a, const Units& u, int G) {
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int Hkv = a.num_kv_heads;
    for (int i = threadIdx.x; i < a.num_seqs * Hkv; i += blockDim.x) a.parts[i] = PrefixParts{0, 0, 0, 0};
    __syncthreads();
    if (u.W == 0) return;
    int tile0 = 0, row0 = 0;
    bool bad = false;
    for (int g0 = 0; g0 < a.num_groups; g0 += 32) {
        const GroupShape p = g0 == 0 ? u.first : group_shape(a, g0 + lane, G, &bad);
        const int work = group_work(p, Hkv);
        const int parts = mul_div(p.keys, u.P, u.W) + 2;
        const int rows = p.keys ? Hkv * parts * p.rows : 0;
        for (int k = 0; k < 32; ++k) {  // the groups one after the other, a warp's share of the pairs each
            const int n = __shfl_sync(0xffffffffu, work, k);
            const int keys = __shfl_sync(0xffffffffu, p.keys, k), tiles = __shfl_sync(0xffffffffu, p.tiles, k);
            const int grows = __shfl_sync(0xffffffffu, p.rows, k), seq0 = __shfl_sync(0xffffffffu, p.seq0, k);
            const int np = __shfl_sync(0xffffffffu, parts, k), blocks = __shfl_sync(0xffffffffu, p.blocks, k);
            const int reserved = __shfl_sync(0xffffffffu, rows, k);
            const int pairs = n ? grows / G * Hkv : 0;
            for (int i = warp * 32 + lane; i < pairs; i += warps * 32) {
                const int s = i / Hkv, h = i - s * Hkv;
                if (a.context_lens[seq0 + s] / a.block_size < blocks) continue;  // ends inside the prefix
                const int rt = s * G >> 7;
                const int first = tile0 + (h * tiles + rt) * keys;
                const int ca = cta_of_tile(first, u.W, u.P), cb = cta_of_tile(first + keys - 1, u.W, u.P);
                a.parts[static_cast<int64_t>(seq0 + s) * Hkv + h] =
                    PrefixParts{row0 + h * np * grows + s * G, grows, cb - ca + 1, 0};
            }
            tile0 += n;
            row0 += reserved;
        }
    }
}

// ------------------------------------------------------------------ parts

constexpr int kBM = 128;            // rows a CTA
constexpr int kNK = kPrefixTile;    // keys a tile
constexpr uint32_t kTmemCols = 256; // S / P buffers (2 x 64) + O (head_dim)
constexpr float kLazy = 8.f;

template <int D, bool kFP8>
struct Shape {
    static constexpr int kSlices = D / 64;                    // 128-byte slices of a row
    static constexpr int kKRing = D == 128 ? 3 : 6;           // K stages
    static constexpr int kVRing = D == 128 ? 2 : 4;           // V stages
    static constexpr uint32_t kTile = kSlices * kNK * 128;    // bytes of a K (or V) tile
    static constexpr int kProducers = kFP8 ? 4 : 1;           // producer warps
    static constexpr int kThreads = 32 * (5 + kProducers);
    static constexpr int kCtas = kFP8 ? 1 : 2;                // CTAs an SM
    // E4M3: codes on their way, a ring for each producer warp: its 16 rows of K and of V.
    static constexpr int kRawRing = kFP8 ? 6 : 0;
    static constexpr uint32_t kRawStage = 2 * 16 * 128;
    static constexpr uint32_t kQOff = 0;
    static constexpr uint32_t kKOff = kSlices * kBM * 128;
    static constexpr uint32_t kVOff = kKOff + kKRing * kTile;
    static constexpr uint32_t kRawOff = kVOff + kVRing * kTile;
    static constexpr uint32_t kBarOff = kRawOff + kProducers * kRawRing * kRawStage;
};

struct Bars {
    uint64_t kfull[6], kempty[6], vfull[4], vempty[4];
    uint64_t s_full[2], p_full[2], pv_done[2], q_full;
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

// Eight E4M3 codes -> eight f16 values, exactly, times 2^-8.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
    return make_uint4(e4m3x2_odd_bytes_to_half2_shifted(__byte_perm(lo, 0u, 0x1404)),
                      e4m3x2_odd_bytes_to_half2_shifted(__byte_perm(lo, 0u, 0x3424)),
                      e4m3x2_odd_bytes_to_half2_shifted(__byte_perm(hi, 0u, 0x1404)),
                      e4m3x2_odd_bytes_to_half2_shifted(__byte_perm(hi, 0u, 0x3424)));
}

// QT: q's type.  The tensor cores work in it, or in f16 over an E4M3 cache
// (whose codes widen to f16 in a few integer operations); a bf16 q is then
// brought to f16 with a power of two for each row that puts its largest
// element at 2^13: exact down to 2^-27 of that element.
template <int QT, int D, bool kFP8>
__global__ void __launch_bounds__(Shape<D, kFP8>::kThreads, Shape<D, kFP8>::kCtas)
    shared_prefix_parts_kernel(const SharedPrefixArgs a) {
    using T = typename Elem<QT>::T;
    using S = Shape<D, kFP8>;
    constexpr int DT = kFP8 ? static_cast<int>(kF16) : QT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    pdl_wait();
    pdl_allow_next();  // after the wait: the tails start when all that came before has completed
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.num_q_heads / a.num_kv_heads;
    const Units units = plan_units(a, G);
    const int cta = blockIdx.x;
    if (cta == static_cast<int>(gridDim.x) - 1) {  // the last CTA has no tiles
        write_parts_table(a, units, G);
        return;
    }
    if (units.W == 0 || cta >= units.P) return;
    const int start = mul_div(cta, units.W, units.P), end = mul_div(cta + 1, units.W, units.P);
    // The swizzled layouts need a 1024-byte aligned base.
    if (smem_addr(smem_raw) & 1023u) {
        if (tid == 0) raise_flag(a.status, kFlagBadPlan);
        return;
    }
    uint8_t* base = smem_raw;
    Bars* B = reinterpret_cast<Bars*>(base + S::kBarOff);
    volatile int* abort = &B->abort;
    if (tid == 0) {
        constexpr int arrivals = kFP8 ? S::kProducers : 32;  // one a producer warp, or one a copying lane
        for (int i = 0; i < S::kKRing; ++i) {
            mbar_init(&B->kfull[i], arrivals);
            mbar_init(&B->kempty[i], 1);
        }
        for (int i = 0; i < S::kVRing; ++i) {
            mbar_init(&B->vfull[i], arrivals);
            mbar_init(&B->vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B->s_full[i], 1);
            mbar_init(&B->p_full[i], 4);
            mbar_init(&B->pv_done[i], 1);
        }
        mbar_init(&B->q_full, 4);
        B->abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) tc_alloc(&B->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = B->tmem;

    // Every role walks the CTA's segments; tiles are counted from the CTA's
    // first (i), so rings and buffers go on over segments.
    if (warp >= 5) {
        // ---- producers: K of tile i, then V of tile i - 1 (K runs one tile
        // ahead: S of a tile is issued before its PV).  The keys come in runs
        // of 16 (block_size is a multiple of 16), each inside one block; runs
        // past the last key are zeros.
        const int bs = a.block_size;
        const int ch = lane & 7, l8 = lane >> 3;
        int i = 0;  // K tiles asked for so far
        bool ok = true;
        [[maybe_unused]] const uint32_t sw0 = static_cast<uint32_t>(ch ^ l8) << 4, sw1 = static_cast<uint32_t>(ch ^ (l8 + 4)) << 4;
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
            auto run_row = [&](int r) -> int64_t {
                if (r >= nruns || lead < 0) return -1;
                const int key = key0 + 16 * r;
                const int lb = key / bs;
                int blk = table[lb];
                if (blk < 0 || blk >= a.num_blocks) {
                    raise_flag(a.status, kFlagBadBlock);
                    blk = 0;
                }
                return (static_cast<int64_t>(blk) * a.num_kv_heads + t.h) * bs + (key - lb * bs);
            };
            if constexpr (!kFP8) {
                // Lane l knows where run l of the current 8 tiles starts, and
                // of the 8 after them.
                int64_t now = run_row(lane), next = run_row(32 + lane);
                // Lane e copies chunk e % 8 of rows e / 8 + 4 q of a run.
                auto load = [&](int j, int64_t rows, const void* cache, uint32_t dst, uint64_t* bar) {
                    const char* c0 = static_cast<const char*>(cache) + l8 * (D * 2) + ch * 16;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t row = __shfl_sync(0xffffffffu, rows, (j & 7) * 4 + k);
                        const bool real = row >= 0;
                        const char* src = c0 + (real ? row : 0) * (D * 2);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t d = dst + (16 * k + 4 * q + l8) * 128 + ((q & 1) ? sw1 : sw0);
#pragma unroll
                            for (int sl = 0; sl < S::kSlices; ++sl)
                                cp_async_16_or_zero(d + sl * (kNK * 128), src + (real ? q * (4 * D * 2) + sl * 128 : 0), real);
                        }
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
                };
                int64_t before = now;
                for (int j = 0; j <= n && ok; ++j) {
                    if (j < n) {
                        const int st = (i + j) % S::kKRing;
                        if ((j & 7) == 0 && j > 0) {
                            before = now;
                            now = next;
                            next = run_row(4 * (j + 8) + lane);
                        }
                        if (i + j >= S::kKRing)
                            ok = __all_sync(0xffffffffu, wait(&B->kempty[st], (i + j) / S::kKRing - 1, abort, a.status));
                        if (!ok) break;
                        load(j, now, a.k_cache, smem_addr(base + S::kKOff + st * S::kTile), &B->kfull[st]);
                    }
                    if (j >= 1) {
                        const int v = i + j - 1, st = v % S::kVRing;
                        if (v >= S::kVRing)
                            ok = __all_sync(0xffffffffu, wait(&B->vempty[st], v / S::kVRing - 1, abort, a.status));
                        if (!ok) break;
                        load(j - 1, (j & 7) == 0 && j < n ? before : now, a.v_cache,
                             smem_addr(base + S::kVOff + st * S::kTile), &B->vfull[st]);
                    }
                }
            } else {
                // E4M3: warp w brings run w of every tile: its codes travel
                // through a ring of its own (asynchronous copies, each lane
                // reading back what it copied) and are widened into the tile.
                // Lane e takes codes 16 (e % 8) .. of rows e / 8 + 4 q.
                const int w = warp - 5;
                const uint32_t raw0 = smem_addr(base + S::kRawOff + w * (S::kRawRing * S::kRawStage)) + lane * 16;
                int64_t rows = -1;  // lane l: run w of tile l of the current 32
                auto ask = [&](int j) {
                    if ((j & 31) == 0) rows = run_row(4 * (j + lane) + w);
                    const int64_t row = __shfl_sync(0xffffffffu, rows, j & 31);
                    if (j < n) {
                        const bool real = row >= 0;
                        const int64_t off = real ? (row + l8) * D + ch * 16 : 0;
                        const uint32_t d = raw0 + (j % S::kRawRing) * S::kRawStage;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            cp_async_16_or_zero(d + q * 512, static_cast<const char*>(a.k_cache) + off + (real ? q * 4 * D : 0), real);
                            cp_async_16_or_zero(d + 2048 + q * 512, static_cast<const char*>(a.v_cache) + off + (real ? q * 4 * D : 0), real);
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");  // an empty group past the end
                };
                auto put = [&](uint32_t raw, uint32_t off, uint64_t* bar) {
                    uint8_t* tile = base + off + (ch >> 2) * (kNK * 128);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 r;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                                     : "r"(raw + q * 512)
                                     : "memory");
                        const int row = 16 * w + 4 * q + l8;
                        const int c0 = (ch & 3) * 2;
                        *reinterpret_cast<uint4*>(tile + row * 128 + ((c0 ^ (row & 7)) << 4)) = widen8(r.x, r.y);
                        *reinterpret_cast<uint4*>(tile + row * 128 + (((c0 + 1) ^ (row & 7)) << 4)) = widen8(r.z, r.w);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                };
                for (int j = 0; j < S::kRawRing - 1; ++j) ask(j);
                for (int j = 0; j < n && ok; ++j) {
                    ask(j + S::kRawRing - 1);
                    asm volatile("cp.async.wait_group %0;" ::"n"(S::kRawRing - 1) : "memory");  // tile j is here
                    const uint32_t raw = raw0 + (j % S::kRawRing) * S::kRawStage;
                    const int sk = (i + j) % S::kKRing, sv = (i + j) % S::kVRing;
                    if (i + j >= S::kKRing)
                        ok = __all_sync(0xffffffffu, wait(&B->kempty[sk], (i + j) / S::kKRing - 1, abort, a.status));
                    if (!ok) break;
                    put(raw, S::kKOff + sk * S::kTile, &B->kfull[sk]);
                    if (i + j >= S::kVRing)
                        ok = __all_sync(0xffffffffu, wait(&B->vempty[sv], (i + j) / S::kVRing - 1, abort, a.status));
                    if (!ok) break;
                    put(raw + 2048, S::kVOff + sv * S::kTile, &B->vfull[sv]);
                }
            }
            i += n;
            x += n;
        }
        // Every copy issued must land before the CTA can exit.
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp == 4) {
        // ---- MMA issue (one lane; the others only look segments up)
        constexpr int bf = DT == kBF16 ? 1 : 0;
        constexpr uint32_t idS = tc_idesc_f16(bf, false, kNK, kBM);
        constexpr uint32_t idPV = tc_idesc_f16(bf, true, D, kBM);
        const uint32_t qa = smem_addr(base + S::kQOff);
        auto pv = [&](int i, bool first) -> bool {
            const int sv = i % S::kVRing, bt = i & 1;
            if (!wait(&B->p_full[bt], i >> 1, abort, a.status)) return false;
            if (!wait(&B->vfull[sv], i / S::kVRing, abort, a.status)) return false;
            if constexpr (!kFP8) fence_proxy_async_smem();  // lane copies before the tensor cores read them
            tc_fence_after();
            const uint32_t va = smem_addr(base + S::kVOff + sv * S::kTile);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < kNK / 16; ++kk)
                    tc_mma_ts(taddr + 128, taddr + bt * kNK + part * 32 + kk * 8,
                              tc_sdesc(va + kk * 16 * 128, kNK * 128, 1024), idPV, !(first && part == 0 && kk == 0));
            tc_commit(&B->pv_done[bt]);
            tc_commit(&B->vempty[sv]);
            return true;
        };
        int i = 0, seg = 0;
        bool ok = true;
        for (int x = start; x < end && ok; ++seg) {
            const Triple t = find_triple(a, units, G, x);
            const int n = min(end, t.tile0 + t.keys) - x;
            if (lane == 0) {
                ok = wait(&B->q_full, seg, abort, a.status);
                for (int j = 0; j < n && ok; ++j) {
                    const int k = i + j, sk = k % S::kKRing, b = k & 1;
                    ok = wait(&B->kfull[sk], k / S::kKRing, abort, a.status);
                    // S buffer b holds P of tile k - 2 until that PV has completed.
                    if (ok && k >= 2) ok = wait(&B->pv_done[b], (k >> 1) - 1, abort, a.status);
                    if (!ok) break;
                    if constexpr (!kFP8) fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t ka = smem_addr(base + S::kKOff + sk * S::kTile);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc_mma(taddr + b * kNK, tc_sdesc(qa + (ks >> 2) * (kBM * 128) + (ks & 3) * 32, 16, 1024),
                               tc_sdesc(ka + (ks >> 2) * (kNK * 128) + (ks & 3) * 32, 16, 1024), idS, ks > 0);
                    tc_commit(&B->s_full[b]);
                    tc_commit(&B->kempty[sk]);
                    if (j >= 1) ok = pv(k - 1, j == 1);
                }
                if (ok) ok = pv(i + n - 1, n == 1);
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            i += n;
            x += n;
        }
    } else {
        // ---- softmax: thread r owns row r (tensor-memory lane r)
        const int r = tid;
        const uint32_t lane_base = taddr + (static_cast<uint32_t>(32 * warp) << 16);
        // |scale| in log2 units; a zero scale is taken as 1e-30, which leaves
        // every finite score's exponent at 0 while masked scores stay -inf.
        const float sc0 = fmaxf(fabsf(a.scale_log2), 1e-30f) * (kFP8 ? 256.f : 1.f);  // widened codes are 2^-8 of the value
        int i = 0;
        bool ok = true;
        for (int x = start; x < end && ok;) {
            const Triple t = find_triple(a, units, G, x);
            const int n = min(end, t.tile0 + t.keys) - x;
            const int nrows = min(kBM, t.rows - t.rt * kBM);
            const int keys = min(t.blocks * a.block_size - (x - t.tile0) * kNK, n * kNK);  // of the segment
            float sc = sc0;
            {
                // Q row r of the tile (member (rt * 128 + r) / G, query head
                // h * G + r % G) into shared memory, 128-byte swizzled K-major.
                // (The previous segment's S are complete: their last was read.)
                const int rr = t.rt * kBM + min(r, nrows - 1);
                const T* qrow = static_cast<const T*>(a.q) +
                                (static_cast<int64_t>(t.seq0 + rr / G) * a.num_q_heads + t.h * G + rr % G) * D;
                // A negative scale is applied as |scale| to the scores of -q (a
                // sign flip is exact), so the row maximum is taken on unscaled
                // scores.
                const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
                float up = 1.f;
                if constexpr (kFP8 && QT == kBF16) {
                    uint32_t top = 0;  // largest |q|, as the bits of a bf16
#pragma unroll
                    for (int q16 = 0; q16 < D / 8; ++q16) {
                        const uint4 v = *reinterpret_cast<const uint4*>(qrow + 8 * q16);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
                    }
                    const int e = min(max(static_cast<int>(top >> 7) - 127, -100), 127);  // its exponent
                    up = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
                    sc *= __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
                }
#pragma unroll
                for (int q16 = 0; q16 < D / 8; ++q16) {
                    uint4 v = *reinterpret_cast<const uint4*>(qrow + 8 * q16);
                    if constexpr (kFP8 && QT == kBF16) {
                        uint32_t* w = &v.x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __half2 h = __floats2half2_rn(__uint_as_float(w[k] << 16) * up,
                                                                __uint_as_float(w[k] & 0xFFFF0000u) * up);
                            w[k] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
                    v.x ^= flip;
                    v.y ^= flip;
                    v.z ^= flip;
                    v.w ^= flip;
                    *reinterpret_cast<uint4*>(base + S::kQOff + (q16 >> 3) * (kBM * 128) + r * 128 +
                                              (((q16 & 7) ^ (r & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->q_full);  // one arrival per warp (count 4)
            }
            float m_ref = 0.f, l = 0.f;
            for (int j = 0; j < n && ok; ++j) {
                const int k0 = i + j, b = k0 & 1;
                ok = __all_sync(0xffffffffu, wait(&B->s_full[b], k0 >> 1, abort, a.status));
                if (!ok) break;
                tc_fence_after();
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
                for (int k = 0; k < 8; ++k) mx[k] = sv[k];
#pragma unroll
                for (int k = 8; k < kNK; ++k) mx[k & 7] = fmaxf(mx[k & 7], sv[k]);
                // (The lower limit keeps the exponents of a row whose scores
                // are all -inf so far at -inf, not NaN.)
                const float mt = fmaxf(fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                             fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sc,
                                       -1e30f);
                bool need = false;
                if (j == 0)
                    m_ref = mt;
                else
                    need = mt > m_ref + kLazy;
                if (__any_sync(0xffffffffu, need)) {
                    // O must be complete up to the tile before it is rescaled.
                    ok = __all_sync(0xffffffffu, wait(&B->pv_done[(k0 - 1) & 1], (k0 - 1) >> 1, abort, a.status));
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
                        tc_ld32(lane_base + 128 + 32 * cb, o);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= f;
                        tc_st32(lane_base + 128 + 32 * cb, o);
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
            if (ok) ok = __all_sync(0xffffffffu, wait(&B->pv_done[(i - 1) & 1], (i - 1) >> 1, abort, a.status));
            if (ok) {
                tc_fence_after();
                const float vs = a.v_scale * (kFP8 ? 256.f : 1.f);
                const int64_t row = t.row0 + static_cast<int64_t>(cta - cta_of_tile(t.tile0, units.W, units.P)) * t.stride + r;
                const bool row_ok = r < nrows && row < a.max_rows;
                float* po = a.part_o + row * D;
#pragma unroll
                for (int cb = 0; cb < D / 32; ++cb) {
                    float o[32];
                    tc_ld32(lane_base + 128 + 32 * cb, o);
                    tc_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= vs;
#pragma unroll
                        for (int k = 0; k < 32; k += 8) store_32(po + 32 * cb + k, o + k);
                    }
                }
                if (row_ok) *reinterpret_cast<float2*>(a.part_ml + 2 * row) = make_float2(m_ref, l);
                tc_fence_before();  // before the next segment's P, and its PV, are announced
            }
            x += n;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc_dealloc(taddr, kTmemCols);
    }
}

// ------------------------------------------------------------------ merge

// One warp a (sequence, query head): the prefix's parts, then the parts the
// decode kernel left of the tail.  Lane l holds (max, sum) of part l of 32;
// every lane sums D / 32 output elements.
template <int D>
__global__ void __launch_bounds__(128) shared_prefix_merge_kernel(const SharedPrefixArgs a, const DecodeArgs d) {
    constexpr int VD = D / 32;
    pdl_allow_next();
    pdl_wait();
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (row >= static_cast<int64_t>(a.num_seqs) * a.num_q_heads) return;
    const int s = static_cast<int>(row / a.num_q_heads);
    const int hq = static_cast<int>(row - static_cast<int64_t>(s) * a.num_q_heads);
    const int G = a.num_q_heads / a.num_kv_heads;
    const int h = hq / G, g = hq - h * G;
    const int Hc = d.heads_per_stage, chunks = d.num_kv_heads / Hc;
    const int hc = h / Hc, hw = h - hc * Hc;
    const int pair = s * chunks + hc;
    const PrefixParts pp = a.parts[s * a.num_kv_heads + h];
    const int4 tp = d.tail_parts[pair];
    const int n = pp.parts + tp.y;
    float M = -INFINITY, L = 0.f, acc[VD];
#pragma unroll
    for (int i = 0; i < VD; ++i) acc[i] = 0.f;
    for (int base = 0; base < n; base += 32) {
        // This lane's part: its (max, sum) and its outputs.
        const int p = base + lane;
        const float* po = nullptr;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (p < pp.parts) {
            const int64_t r = pp.row0 + static_cast<int64_t>(p) * pp.stride + g;
            if (r < a.max_rows) {
                po = a.part_o + r * D;
                ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + 2 * r));
            }
        } else if (p < n) {
            const int k = p - pp.parts;
            const int64_t c = tp.w == 0 ? tp.x + k : cta_of_tile(tp.z + k, tp.w, d.num_ctas);
            const int64_t r = ((c + pair) * Hc + hw) * G + g;
            po = d.part_o + r * D;
            ml = __ldcg(reinterpret_cast<const float2*>(d.part_ml + 2 * r));
        }
        const uint64_t addr = reinterpret_cast<uint64_t>(po);
        const int cnt = min(32, n - base);
        // Outputs of eight parts; the first eight are asked for together with
        // the (max, sum) pairs.
        float v[8][VD];
        auto fetch = [&](int k0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, addr, (k0 + k) & 31));
                const bool get = k0 + k < cnt && src != nullptr;
                if constexpr (VD == 4) {
                    const float4 t = get ? __ldcg(reinterpret_cast<const float4*>(src) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[k][0] = t.x, v[k][1] = t.y, v[k][2] = t.z, v[k][3] = t.w;
                } else {
                    const float2 t = get ? __ldcg(reinterpret_cast<const float2*>(src) + lane) : make_float2(0.f, 0.f);
                    v[k][0] = t.x, v[k][1] = t.y;
                }
            }
        };
        fetch(0);
        float mx = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float Mn = fmaxf(M, mx);
        const float w = po ? fast_exp2(ml.x - Mn) : 0.f;
        const float al = base == 0 ? 0.f : fast_exp2(M - Mn);
        float ls = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        L = L * al + ls;
        M = Mn;
#pragma unroll
        for (int i = 0; i < VD; ++i) acc[i] *= al;
        for (int k0 = 0; k0 < cnt; k0 += 8) {
            if (k0 > 0) fetch(k0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                if (k0 + k < cnt) {
#pragma unroll
                    for (int i = 0; i < VD; ++i) acc[i] = fmaf(wk, v[k][i], acc[i]);
                }
            }
        }
    }
    const float inv = n > 0 ? 1.f / L : 0.f;  // a sequence without tokens: zeros
    const int64_t o0 = row * D + lane * VD;
#pragma unroll
    for (int i = 0; i < VD; ++i) store_out(a.out, o0 + i, n > 0 ? acc[i] * inv : 0.f, a.out_dtype);
}

template <int DT, int D, bool kFP8>
cudaError_t launch_parts_t(const SharedPrefixArgs& a, cudaStream_t stream) {
    using S = Shape<D, kFP8>;
    static std::atomic<int> configured[64];
    auto kern = shared_prefix_parts_kernel<DT, D, kFP8>;
    const bool cacheable = a.device >= 0 && a.device < 64;
    if (!cacheable || !configured[a.device].load()) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, a.smem_bytes);
        if (e != cudaSuccess) return e;
        if (cacheable) configured[a.device].store(1);
    }
    return launch_kernel(kern, dim3(a.num_sms * a.ctas_per_sm + 1), dim3(S::kThreads), static_cast<size_t>(a.smem_bytes), stream, true, a);
}

}  // namespace

int prefix_smem_bytes(int head_dim, bool fp8) {
    const uint32_t off = fp8 ? Shape<128, true>::kBarOff : head_dim == 64 ? Shape<64, false>::kBarOff : Shape<128, false>::kBarOff;
    return static_cast<int>(off + sizeof(Bars));
}

int prefix_ctas_per_sm(bool fp8) { return fp8 ? Shape<128, true>::kCtas : Shape<128, false>::kCtas; }

cudaError_t launch_prefix_parts(const SharedPrefixArgs& a, cudaStream_t stream) {
    if (a.kv_dtype == kFP8) {
        if (a.dtype == kBF16) return launch_parts_t<kBF16, 128, true>(a, stream);
        return launch_parts_t<kF16, 128, true>(a, stream);
    }
    if (a.head_dim == 64) {
        if (a.dtype == kBF16) return launch_parts_t<kBF16, 64, false>(a, stream);
        return launch_parts_t<kF16, 64, false>(a, stream);
    }
    if (a.dtype == kBF16) return launch_parts_t<kBF16, 128, false>(a, stream);
    return launch_parts_t<kF16, 128, false>(a, stream);
}

cudaError_t launch_prefix_merge(const SharedPrefixArgs& a, const DecodeArgs& tails, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
    const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
    if (a.head_dim == 64) return launch_kernel(shared_prefix_merge_kernel<64>, grid, dim3(128), 0, stream, true, a, tails);
    return launch_kernel(shared_prefix_merge_kernel<128>, grid, dim3(128), 0, stream, true, a, tails);
}

}  // namespace pkv
