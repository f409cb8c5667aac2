// How the shared-prefix attention (shared_prefix_kernel.cuh) divides its work,
// worked out alike by every CTA from the groups and lengths.
//
// The prefix part's work is key tiles: every (group, KV head, row tile) triple
// has its group's tiles, triples in that order.  CTA c of P takes tiles
// [c W / P, (c + 1) W / P), whatever triples they belong to: all CTAs have the
// same work to within a tile.  A run of one triple's tiles in one CTA is a
// segment, and leaves one part.  Part k of a triple comes from the k-th CTA
// that has tiles of it; a group reserves keys P / W + 2 parts of each of its
// rows, so all groups together reserve at most 128 P + 2 (all rows).
//
// The SMs are divided between the two roles, one CTA on each, so that they run
// side by side and end together.
#pragma once

#include "device_utils.cuh"

namespace pkv {

constexpr int kPrefixRows = 128;  // query rows of a row tile
constexpr int kPrefixTile = 64;   // keys of a tile

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

// Group g's shape; no work for one past the last.  *bad: it is out of order.
// (Args: SharedPrefixArgs or DecodeArgs.)
template <class Args>
__device__ __forceinline__ GroupShape group_shape(const Args& a, int g, int G, bool* bad) {
    GroupShape p{0, 0, 0, 0, 0};
    if (g >= a.num_groups) return p;
    const int s0 = a.group_start[g], s1 = a.group_start[g + 1], len = a.prefix_lens[g];
    if (s0 < 0 || s1 > a.num_seqs || s0 > s1 || len < 0) {
        *bad = true;
        return p;
    }
    p.seq0 = s0;
    p.rows = (s1 - s0) * G;
    p.tiles = (p.rows + kPrefixRows - 1) / kPrefixRows;
    p.blocks = len / a.block_size;
    if (p.blocks > a.max_blocks) p.blocks = 0;  // no sequence is that long
    p.keys = (p.blocks * a.block_size + kPrefixTile - 1) / kPrefixTile;
    return p;
}

// Blocks that sequence s, of ctx tokens, shares with its group: 0 if it is in
// none, or ends inside them.  The groups are in order.
template <class Args>
__device__ __forceinline__ int shared_blocks(const Args& a, int s, int ctx) {
    if (a.num_groups == 0) return 0;
    int lo = 0, hi = a.num_groups;  // the last group that starts at or before s
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.group_start[mid] <= s)
            lo = mid;
        else
            hi = mid;
    }
    const int n = a.prefix_lens[lo] / a.block_size;
    return a.group_start[lo] <= s && s < a.group_start[lo + 1] && n <= ctx / a.block_size ? n : 0;
}

// What every warp works out alike.
struct Units {
    GroupShape first;  // this lane's group of the first 32
    int W;             // tiles; 0: nothing is shared
    int triples;       // (group, KV head, row tile) triples with tiles
    bool bad;          // the groups are out of order
    int P;             // CTAs of the parts role (divide_sms)
};

template <class Args>
__device__ __forceinline__ Units plan_units(const Args& a, int G) {
    const int lane = threadIdx.x & 31;
    Units u;
    bool bad = false;
    u.first = group_shape(a, lane, G, &bad);
    int work = a.num_kv_heads * u.first.tiles * u.first.keys, triples = u.first.keys ? u.first.tiles : 0;
    for (int g0 = 32; g0 < a.num_groups; g0 += 32) {
        const GroupShape p = group_shape(a, g0 + lane, G, &bad);
        work += a.num_kv_heads * p.tiles * p.keys;
        triples += p.keys ? p.tiles : 0;
    }
    u.bad = __any_sync(0xffffffffu, bad);
    work = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(work)));
    triples = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(triples))) * a.num_kv_heads;
    u.W = u.bad ? 0 : work;
    u.triples = triples;
    u.P = 0;
    return u;
}

// The parts role's share of the SMs, u->P; the tails take the rest: `items` of
// `tokens` (token, KV head) rows, with phantoms among them (DecodeArgs), of
// `pairs` (sequence, heads of a stage).
//
// Measured costs on one SM, of 128-dim heads and 4 query heads a KV head: a tile
// of the parts role kTileNs (64 dims: their own), the start and end of a triple
// kTripleNs; the tails kTokenNs for each row, whatever its length (the consumer's
// arithmetic or the memory's rate), and kSequenceNs for each pair.  The one figure
// for a tails row is rough for other heads: in a graph, with 0.5 / 0.75 / 1 / 1.5
// times it, 256 sequences over 32,768 shared tokens take 312 / 188 / 190 / 213 us,
// 64 in groups of 8 with long tails 266 / 267 / 269 / 311; 32 over 4,096 with tails
// of 2,048, 4 query heads a KV head and 128 dims 34 / 40 / 38 / 48, with 64 dims 29 /
// 33 / 39 / 46.
template <class Args>
__device__ __forceinline__ void divide_sms(const Args& a, int items, int tokens, int pairs, Units* u) {
    constexpr float kTripleNs = 3000.f, kSequenceNs = 3700.f;
    const bool fp8 = a.kv_dtype == kFP8;
    const float kTileNs = a.head_dim == 64 ? 560.f : fp8 ? 1400.f : 1000.f;
    const float kTokenNs = fp8 ? 7.f : 10.f;
    const int sms = a.num_ctas;
    if (u->W == 0) return;
    const float parts = kTileNs * static_cast<float>(u->W) + kTripleNs * static_cast<float>(u->triples);
    const float tails = kTokenNs * static_cast<float>(max(items - a.phantom * pairs, 0)) * static_cast<float>(tokens) +
                        kSequenceNs * static_cast<float>(pairs);
    int P = static_cast<int>(static_cast<float>(sms) * parts / (parts + tails) + 0.5f);
    P = max(1, min(min(P, u->W), sms - 1));  // a tails CTA there always is: it writes the merge's tables
    // CTAs that begin with a triple have one segment: worth up to a quarter of
    // them while a CTA has few tiles, a sixteenth always.
    if (u->triples <= P) {
        const int even = P / u->triples * u->triples;
        if ((P - even) * (u->W / P < 16 ? 4 : 16) <= P) P = even;
    }
    u->P = P;
}

// A triple, and where its parts go.
struct Triple {
    int seq0, rows, blocks, keys;
    int h, rt;       // KV head, row tile
    int tile0;       // its first tile
    int row0;        // partial row of the row tile's first row, part 0
};

// Tile x of a group whose first tile and partial row are `first` and row0, with
// `parts` parts of each row: its head, row tile and places.
__device__ __forceinline__ void place_in_group(Triple* t, int x, int first, int row0, int tiles, int parts) {
    const int k = (x - first) / t->keys;
    t->h = tiles == 1 ? k : k / tiles;
    t->rt = k - t->h * tiles;
    t->tile0 = first + k * t->keys;
    t->row0 = row0 + t->h * parts * t->rows + t->rt * kPrefixRows;
}

// The triple of tile x, by the whole warp (0 <= x < W).  Part k of row r of its
// row tile is partial row row0 + k * rows + r.
template <class Args>
__device__ __forceinline__ Triple find_triple(const Args& a, const Units& u, int G, int x) {
    const int lane = threadIdx.x & 31;
    Triple t{};
    if (a.num_groups == 1) {
        t.seq0 = __shfl_sync(0xffffffffu, u.first.seq0, 0);
        t.rows = __shfl_sync(0xffffffffu, u.first.rows, 0);
        t.blocks = __shfl_sync(0xffffffffu, u.first.blocks, 0);
        t.keys = __shfl_sync(0xffffffffu, u.first.keys, 0);
        place_in_group(&t, x, 0, 0, (t.rows + kPrefixRows - 1) / kPrefixRows, mul_div(t.keys, u.P, u.W) + 2);
        return t;
    }
    int tile0 = 0, row0 = 0;
    bool bad = false;
    for (int g0 = 0; g0 < a.num_groups; g0 += 32) {
        const GroupShape p = g0 == 0 ? u.first : group_shape(a, g0 + lane, G, &bad);
        const int work = a.num_kv_heads * p.tiles * p.keys;
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
            place_in_group(&t, x, first, row0 + __shfl_sync(0xffffffffu, r - rows, src), tiles, np);
            return t;
        }
        tile0 += __shfl_sync(0xffffffffu, w, 31);
        row0 += __shfl_sync(0xffffffffu, r, 31);
    }
    return t;
}

}  // namespace pkv
