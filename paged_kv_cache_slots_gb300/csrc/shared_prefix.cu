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

constexpr int kMinChunk = 4;  // key tiles, see chunk_tiles

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One lane's group, without its place.
struct GroupShape {
    int seq0, rows, tiles, keys, blocks;  // keys: tiles of kPrefixTile
};

__device__ __forceinline__ GroupShape group_shape(const SharedPrefixArgs& a, int g, int G) {
    GroupShape p{0, 0, 0, 0, 0};
    if (g >= a.num_groups) return p;
    p.seq0 = a.group_start[g];
    p.rows = (a.group_start[g + 1] - p.seq0) * G;
    p.tiles = (p.rows + 127) / 128;
    p.blocks = a.prefix_lens[g] / a.block_size;
    if (p.blocks > a.max_blocks) p.blocks = 0;  // no sequence is that long
    p.keys = static_cast<int>((static_cast<int64_t>(p.blocks) * a.block_size + kPrefixTile - 1) / kPrefixTile);
    return p;
}

// Key tiles a chunk, found alike by every warp that asks (the groups are in order).
//
// All chunks should run at once.  With little work a CTA has an SM to itself,
// and a chunk up to four tiles: below that its start and the merge of its
// partial cost more than its tiles.  With more, two CTAs share an SM.  Where
// rounding chunks up to whole tiles gives more CTAs than fit, chunks grow until
// they do (unless there are more (group, KV head, row tile) triples than that).
__device__ int chunk_tiles(const SharedPrefixArgs& a, int G) {
    const int lane = threadIdx.x & 31;
    const int64_t limit = static_cast<int64_t>(a.num_sms) * a.ctas_per_sm;
    int64_t work = 0, triples = 0;
    const GroupShape first = group_shape(a, lane, G);
    for (int g0 = 0; g0 < a.num_groups; g0 += 32) {
        const GroupShape p = g0 == 0 ? first : group_shape(a, g0 + lane, G);
        work += static_cast<int64_t>(p.tiles) * p.keys;
        triples += p.keys ? p.tiles : 0;
    }
    work = warp_sum64(work) * a.num_kv_heads;
    triples = warp_sum64(triples) * a.num_kv_heads;
    int64_t per = (work + limit - 1) / limit;
    const int64_t alone = (work + a.num_sms - 1) / a.num_sms;
    per = max(per, min(alone, static_cast<int64_t>(kMinChunk)));
    if (per < 1) per = 1;
    if (triples >= limit) return static_cast<int>(per);
    for (;;) {
        int64_t units = 0;
        for (int g0 = 0; g0 < a.num_groups; g0 += 32) {
            const GroupShape p = g0 == 0 ? first : group_shape(a, g0 + lane, G);
            units += static_cast<int64_t>(p.tiles) * ((p.keys + per - 1) / per);
        }
        if (warp_sum64(units) * a.num_kv_heads <= limit) return static_cast<int>(per);
        per += (per + 7) / 8;
    }
}

// Calls visit(group, on this lane) for 32 groups at a time, in order, until it
// returns true (on every lane alike).
template <class F>
__device__ __forceinline__ void place_groups(const SharedPrefixArgs& a, int G, int per, F visit) {
    const int lane = threadIdx.x & 31;
    int unit0 = 0, row0 = 0;
    for (int g0 = 0; g0 < a.num_groups; g0 += 32) {
        const GroupShape p = group_shape(a, g0 + lane, G);
        const int chunks = (p.keys + per - 1) / per;
        const int units = a.num_kv_heads * p.tiles * chunks, rows = a.num_kv_heads * chunks * p.rows;
        int u = units, r = rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int yu = __shfl_up_sync(0xffffffffu, u, o), yr = __shfl_up_sync(0xffffffffu, r, o);
            if (lane >= o) u += yu, r += yr;
        }
        const PrefixGroup grp{unit0 + u - units, row0 + r - rows, p.seq0, p.rows, p.tiles, chunks, p.blocks, g0 + lane};
        if (visit(grp, units)) return;
        unit0 += __shfl_sync(0xffffffffu, u, 31);
        row0 += __shfl_sync(0xffffffffu, r, 31);
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
    static constexpr uint32_t kQOff = 0;
    static constexpr uint32_t kKOff = kSlices * kBM * 128;
    static constexpr uint32_t kVOff = kKOff + kKRing * kTile;
    static constexpr uint32_t kBarOff = kVOff + kVRing * kTile;
    static constexpr int kProducers = kFP8 ? 4 : 1;           // producer warps
    static constexpr int kThreads = 32 * (5 + kProducers);
    static constexpr int kCtas = kFP8 ? 1 : 2;                // CTAs an SM
};

struct Bars {
    uint64_t kfull[6], kempty[6], vfull[4], vempty[4];
    uint64_t s_full[2], p_full[2], pv_done[2];
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

// Eight E4M3 codes -> eight values of DT (exact).
template <int DT>
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
    uint32_t h[4] = {e4m3x2_to_half2(static_cast<uint16_t>(lo)), e4m3x2_to_half2(static_cast<uint16_t>(lo >> 16)),
                     e4m3x2_to_half2(static_cast<uint16_t>(hi)), e4m3x2_to_half2(static_cast<uint16_t>(hi >> 16))};
    if constexpr (DT == kBF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
            h[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

template <int DT, int D, bool kFP8>
__global__ void __launch_bounds__(Shape<D, kFP8>::kThreads, Shape<D, kFP8>::kCtas)
    shared_prefix_parts_kernel(const SharedPrefixArgs a) {
    using T = typename Elem<DT>::T;
    using S = Shape<D, kFP8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    pdl_wait();
    pdl_allow_next();  // after the wait: the tails start when all that came before has completed
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.num_q_heads / a.num_kv_heads;
    if (!groups_in_order(a.group_start, a.prefix_lens, a.num_groups, a.num_seqs, a.status)) {
        // Nothing is shared; the last CTA says so to the merge.
        if (blockIdx.x == gridDim.x - 1)
            for (int s = tid; s < a.num_seqs; s += blockDim.x) a.parts[s] = PrefixParts{0, 0, 0, 0};
        return;
    }
    const int per = chunk_tiles(a, G);
    if (blockIdx.x == gridDim.x - 1) {
        // The last CTA has no unit: it tells the merge where every sequence's parts are.
        if (warp == 0)
            place_groups(a, G, per, [&](const PrefixGroup& g, int) {
                if (g.index < a.num_groups) a.groups[g.index] = g;
                return false;
            });
        __syncthreads();
        for (int s = tid; s < a.num_seqs; s += blockDim.x) {
            const int ctx = min(max(a.context_lens[s], 0), a.max_blocks * a.block_size);
            int g = 0;
            PrefixParts p{0, 0, 0, 0};
            if (shared_blocks(a.group_start, a.prefix_lens, a.num_groups, a.block_size, s, ctx, &g) > 0) {
                const PrefixGroup grp = a.groups[g];
                p.row0 = grp.row0 + (s - grp.seq0) * G;
                p.part_stride = grp.rows;
                p.head_stride = grp.rows * grp.chunks;
                p.parts = grp.chunks;
            }
            a.parts[s] = p;
        }
        return;
    }
    const int x = blockIdx.x;
    PrefixGroup grp;
    grp.chunks = 0;
    place_groups(a, G, per, [&](const PrefixGroup& g, int units) {
        const uint32_t mine = __ballot_sync(0xffffffffu, x >= g.unit0 && x < g.unit0 + units);
        if (!mine) return false;
        const int src = __ffs(mine) - 1;
        grp.unit0 = __shfl_sync(0xffffffffu, g.unit0, src);
        grp.row0 = __shfl_sync(0xffffffffu, g.row0, src);
        grp.seq0 = __shfl_sync(0xffffffffu, g.seq0, src);
        grp.rows = __shfl_sync(0xffffffffu, g.rows, src);
        grp.tiles = __shfl_sync(0xffffffffu, g.tiles, src);
        grp.chunks = __shfl_sync(0xffffffffu, g.chunks, src);
        grp.blocks = __shfl_sync(0xffffffffu, g.blocks, src);
        return true;
    });
    if (grp.chunks == 0) return;  // more CTAs than units
    // The member whose table row names the blocks.
    int lead = -1;
    for (int s0 = 0; s0 * G < grp.rows && lead < 0; s0 += 32) {
        const int s = grp.seq0 + s0 + lane;
        const uint32_t in = __ballot_sync(0xffffffffu, (s0 + lane) * G < grp.rows && a.context_lens[s] / a.block_size >= grp.blocks);
        if (in) lead = grp.seq0 + s0 + __ffs(in) - 1;
    }
    if (lead < 0) return;  // every sequence of the group is shorter
    // The swizzled layouts need a 1024-byte aligned base.
    if (smem_addr(smem_raw) & 1023u) {
        if (tid == 0) raise_flag(a.status, kFlagBadPlan);
        return;
    }
    uint8_t* base = smem_raw;
    Bars* B = reinterpret_cast<Bars*>(base + S::kBarOff);
    volatile int* abort = &B->abort;
    const int u = x - grp.unit0;
    const int rt = u % grp.tiles;  // row tiles of a chunk side by side: they share its K and V in L2
    const int c = (u / grp.tiles) % grp.chunks;
    const int h = u / (grp.tiles * grp.chunks);
    const int nkeys = grp.blocks * a.block_size;
    const int key0 = c * per * kNK;
    const int key1 = min(nkeys, key0 + per * kNK);
    const int nkt = (key1 - key0 + kNK - 1) / kNK;
    const int nrows = min(kBM, grp.rows - rt * kBM);

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
        B->abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) tc_alloc(&B->tmem, kTmemCols);
    // Query row r of the tile: member (rt * 128 + r) / G, query head h * G + r % G.
    auto q_row = [&](int r) {
        const int rr = rt * kBM + min(r, nrows - 1);
        return (static_cast<int64_t>(grp.seq0 + rr / G) * a.num_q_heads + h * G + rr % G);
    };
    if (warp < 4) {  // Q rows into shared memory, 128-byte swizzled K-major
        const int r = tid;
        const T* qrow = static_cast<const T*>(a.q) + q_row(r) * D;
        // A negative scale is applied as |scale| to the scores of -q (a sign
        // flip is exact), so the row maximum is taken on unscaled scores.
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int q16 = 0; q16 < D / 8; ++q16) {
            uint4 v = *reinterpret_cast<const uint4*>(qrow + 8 * q16);
            v.x ^= flip;
            v.y ^= flip;
            v.z ^= flip;
            v.w ^= flip;
            *reinterpret_cast<uint4*>(base + S::kQOff + (q16 >> 3) * (kBM * 128) + r * 128 +
                                      (((q16 & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = B->tmem;

    if (warp >= 5) {
        // ---- producers: K of tile i, then V of tile i - 1 (K runs one tile
        // ahead: S of a tile is issued before its PV).  The keys come in runs
        // of 16 (block_size is a multiple of 16), each inside one block; runs
        // past the last key are zeros.
        const int bs = a.block_size;
        const int32_t* table = a.block_tables + static_cast<int64_t>(lead) * a.max_blocks;
        const int nruns = (key1 - key0) / 16;
        // Element offset of run r's first row, in rows of the cache.
        auto run_row = [&](int r) -> int64_t {
            const int key = key0 + 16 * min(r, nruns - 1);
            const int lb = key / bs;
            int blk = table[lb];
            if (blk < 0 || blk >= a.num_blocks) {
                raise_flag(a.status, kFlagBadBlock);
                blk = 0;
            }
            return (static_cast<int64_t>(blk) * a.num_kv_heads + h) * bs + (key - lb * bs);
        };
        if constexpr (!kFP8) {
            // Lane l knows where run l of the current 8 tiles starts, and of
            // the 8 after them.
            int64_t now = run_row(lane), next = run_row(32 + lane), before = now;
            const int ch = lane & 7, l8 = lane >> 3;
            const uint32_t sw0 = static_cast<uint32_t>(ch ^ l8) << 4, sw1 = static_cast<uint32_t>(ch ^ (l8 + 4)) << 4;
            // Lane e copies chunk e % 8 of rows e / 8 + 4 q of a run.
            auto load = [&](int j, int64_t rows, const void* cache, uint32_t dst, uint64_t* bar) {
                const char* c0 = static_cast<const char*>(cache) + l8 * (D * 2) + ch * 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t row = __shfl_sync(0xffffffffu, rows, (j & 7) * 4 + i);
                    const bool real = 4 * j + i < nruns;
                    const char* src = c0 + row * (D * 2);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t d = dst + (16 * i + 4 * q + l8) * 128 + ((q & 1) ? sw1 : sw0);
#pragma unroll
                        for (int sl = 0; sl < S::kSlices; ++sl)
                            cp_async_16_or_zero(d + sl * (kNK * 128), src + q * (4 * D * 2) + sl * 128, real);
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
            };
            for (int i = 0; i <= nkt; ++i) {
                if (i < nkt) {
                    const int st = i % S::kKRing;
                    if ((i & 7) == 0 && i > 0) {
                        before = now;
                        now = next;
                        next = run_row(4 * (i + 8) + lane);
                    }
                    if (i >= S::kKRing &&
                        !__all_sync(0xffffffffu, wait(&B->kempty[st], i / S::kKRing - 1, abort, a.status)))
                        break;
                    load(i, now, a.k_cache, smem_addr(base + S::kKOff + st * S::kTile), &B->kfull[st]);
                }
                if (i >= 1) {
                    const int j = i - 1, st = j % S::kVRing;
                    if (j >= S::kVRing &&
                        !__all_sync(0xffffffffu, wait(&B->vempty[st], j / S::kVRing - 1, abort, a.status)))
                        break;
                    load(j, (i & 7) == 0 && i < nkt ? before : now, a.v_cache, smem_addr(base + S::kVOff + st * S::kTile),
                         &B->vfull[st]);
                }
            }
            // Every copy issued must land before the CTA can exit.
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            // E4M3: warp w widens run w of every tile, exactly, to q's type.
            // Lane e takes codes 16 (e % 8) .. of rows e / 8 + 4 q; the codes
            // of the next tile are loaded before this one's are stored.
            const int w = warp - 5;
            const int ch = lane & 7, l8 = lane >> 3;
            uint4 kr[2][4], vr[2][4];
            auto fetch = [&](int j, uint4 (&kk)[4], uint4 (&vv)[4]) {
                if (j >= nkt) return;
                const bool real = 4 * j + w < nruns;
                const int64_t off = (run_row(4 * j + w) + l8) * D + ch * 16;
                const char* ks = static_cast<const char*>(a.k_cache) + off;
                const char* vs = static_cast<const char*>(a.v_cache) + off;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    kk[q] = real ? __ldg(reinterpret_cast<const uint4*>(ks + q * 4 * D)) : make_uint4(0, 0, 0, 0);
                    vv[q] = real ? __ldg(reinterpret_cast<const uint4*>(vs + q * 4 * D)) : make_uint4(0, 0, 0, 0);
                }
            };
            auto put = [&](const uint4 (&r)[4], uint32_t off, uint64_t* bar) {
                uint8_t* t = base + off + (ch >> 2) * (kNK * 128);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int row = 16 * w + 4 * q + l8;
                    const int c0 = (ch & 3) * 2;
                    *reinterpret_cast<uint4*>(t + row * 128 + ((c0 ^ (row & 7)) << 4)) = widen8<DT>(r[q].x, r[q].y);
                    *reinterpret_cast<uint4*>(t + row * 128 + (((c0 + 1) ^ (row & 7)) << 4)) = widen8<DT>(r[q].z, r[q].w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
            fetch(0, kr[0], vr[0]);
            bool ok = true;
            for (int i0 = 0; i0 < nkt && ok; i0 += 2) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = i0 + k;
                    if (i >= nkt || !ok) continue;
                    fetch(i + 1, kr[k ^ 1], vr[k ^ 1]);
                    const int sk = i % S::kKRing, sv = i % S::kVRing;
                    if (i >= S::kKRing)
                        ok = __all_sync(0xffffffffu, wait(&B->kempty[sk], i / S::kKRing - 1, abort, a.status));
                    if (!ok) continue;
                    put(kr[k], S::kKOff + sk * S::kTile, &B->kfull[sk]);
                    if (i >= S::kVRing)
                        ok = __all_sync(0xffffffffu, wait(&B->vempty[sv], i / S::kVRing - 1, abort, a.status));
                    if (!ok) continue;
                    put(vr[k], S::kVOff + sv * S::kTile, &B->vfull[sv]);
                }
            }
        }
        __syncwarp();
    } else if (warp == 4) {
        // ---- MMA issue (one lane)
        if (lane == 0) {
            constexpr int bf = DT == kBF16 ? 1 : 0;
            constexpr uint32_t idS = tc_idesc_f16(bf, false, kNK, kBM);
            constexpr uint32_t idPV = tc_idesc_f16(bf, true, D, kBM);
            const uint32_t qa = smem_addr(base + S::kQOff);
            auto pv = [&](int t) -> bool {
                const int sv = t % S::kVRing, bt = t & 1;
                if (!wait(&B->p_full[bt], t >> 1, abort, a.status)) return false;
                if (!wait(&B->vfull[sv], t / S::kVRing, abort, a.status)) return false;
                if constexpr (!kFP8) fence_proxy_async_smem();  // lane copies before the tensor cores read them
                tc_fence_after();
                const uint32_t va = smem_addr(base + S::kVOff + sv * S::kTile);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < kNK / 16; ++kk)
                        tc_mma_ts(taddr + 128, taddr + bt * kNK + part * 32 + kk * 8,
                                  tc_sdesc(va + kk * 16 * 128, kNK * 128, 1024), idPV,
                                  !(t == 0 && part == 0 && kk == 0));
                tc_commit(&B->pv_done[bt]);
                tc_commit(&B->vempty[sv]);
                return true;
            };
            bool ok = true;
            for (int j = 0; j < nkt && ok; ++j) {
                const int sk = j % S::kKRing, b = j & 1;
                ok = wait(&B->kfull[sk], j / S::kKRing, abort, a.status);
                // S buffer b holds P of tile j - 2 until that PV has completed.
                if (ok && j >= 2) ok = wait(&B->pv_done[b], (j >> 1) - 1, abort, a.status);
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
                if (j >= 1) ok = pv(j - 1);
            }
            if (ok) pv(nkt - 1);
        }
        __syncwarp();
    } else {
        // ---- softmax: thread r owns row r (tensor-memory lane r)
        const int r = tid;
        const uint32_t lane_base = taddr + (static_cast<uint32_t>(32 * warp) << 16);
        float m_ref = 0.f, l = 0.f;
        // |scale| in log2 units; a zero scale is taken as 1e-30, which leaves
        // every finite score's exponent at 0 while masked scores stay -inf.
        const float sc = fmaxf(fabsf(a.scale_log2), 1e-30f);
        bool ok = true;
        for (int j = 0; j < nkt && ok; ++j) {
            const int b = j & 1;
            ok = __all_sync(0xffffffffu, wait(&B->s_full[b], j >> 1, abort, a.status));
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
            const int left = key1 - key0 - j * kNK;  // keys from this tile on
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
            // (The lower limit keeps the exponents of a row whose scores are
            // all -inf so far at -inf, not NaN.)
            const float mt = fmaxf(fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                         fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sc,
                                   -1e30f);
            bool need = false;
            if (j == 0)
                m_ref = mt;
            else
                need = mt > m_ref + kLazy;
            if (__any_sync(0xffffffffu, need)) {
                // O must be complete up to tile j-1 before it is rescaled.
                ok = __all_sync(0xffffffffu, wait(&B->pv_done[(j - 1) & 1], (j - 1) >> 1, abort, a.status));
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
        if (__all_sync(0xffffffffu, ok && !*abort)) {
            ok = __all_sync(0xffffffffu, wait(&B->pv_done[(nkt - 1) & 1], (nkt - 1) >> 1, abort, a.status));
            tc_fence_after();
            const int64_t row = grp.row0 + (static_cast<int64_t>(h) * grp.chunks + c) * grp.rows + rt * kBM + r;
            const bool row_ok = ok && r < nrows && row < a.max_rows;
            float* po = a.part_o + row * D;
#pragma unroll
            for (int cb = 0; cb < D / 32; ++cb) {
                float o[32];
                tc_ld32(lane_base + 128 + 32 * cb, o);
                tc_wait_ld();
                if (row_ok) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<float4*>(po + 32 * cb + k) =
                            make_float4(o[k] * a.v_scale, o[k + 1] * a.v_scale, o[k + 2] * a.v_scale, o[k + 3] * a.v_scale);
                }
            }
            if (row_ok) *reinterpret_cast<float2*>(a.part_ml + 2 * row) = make_float2(m_ref, l);
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
    const PrefixParts pp = a.num_groups > 0 ? a.parts[s] : PrefixParts{0, 0, 0, 0};
    // The tail's parts: the CTAs that hold its blocks (see decode_plan.cu).
    const int Hc = d.heads_per_stage, chunks = d.num_kv_heads / Hc;
    const int hc = h / Hc, hw = h - hc * Hc;
    const int items = (d.cum[s + 1] - d.cum[s]) / chunks;
    const int nb = items > 0 ? items - d.phantom : 0;
    const int64_t W = d.cum[d.num_seqs], P = d.num_ctas;
    const int64_t first = d.cum[s] + static_cast<int64_t>(hc) * items + d.phantom;
    const int ca = nb > 0 ? cta_of_item(first, W, d.num_ctas) : 0;
    const int cb = nb > 0 ? cta_of_item(first + nb - 1, W, d.num_ctas) : -1;
    const int pair = s * chunks + hc;
    const int n = pp.parts + (cb - ca + 1);
    float M = -INFINITY, L = 0.f, acc[VD];
#pragma unroll
    for (int i = 0; i < VD; ++i) acc[i] = 0.f;
    for (int base = 0; base < n; base += 32) {
        // This lane's part: its (max, sum) and its outputs.
        const int p = base + lane;
        const float* po = nullptr;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (p < pp.parts) {
            const int64_t r = pp.row0 + static_cast<int64_t>(h) * pp.head_stride + static_cast<int64_t>(p) * pp.part_stride + g;
            if (r < a.max_rows) {
                po = a.part_o + r * D;
                ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + 2 * r));
            }
        } else if (p < n) {
            const int64_t c = ca + (p - pp.parts);
            if (!cta_is_empty(c, W, P)) {
                const int64_t r = ((c + pair) * Hc + hw) * G + g;
                po = d.part_o + r * D;
                ml = __ldcg(reinterpret_cast<const float2*>(d.part_ml + 2 * r));
            }
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
    return launch_kernel(kern, dim3(a.max_units + 1), dim3(S::kThreads), static_cast<size_t>(a.smem_bytes), stream, true, a);
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
