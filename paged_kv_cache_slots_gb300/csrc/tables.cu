// Block tables, slots and positions of a step, built on the GPU from how many
// tokens each sequence brings ("vLLM Architecture and Installation", Example 3: a
// sequence takes a block from the front of the free queue when a token crosses a
// block boundary), and blocks given back to the end of the queue.
//
// Extending, for sequences s in order, c_s tokens cached and n_s new:
//   need_s = ceil((c_s + n_s) / bs) - ceil(c_s / bs),  N_s = sum of need up to s,
//   T_s = sum of n up to s;  s is granted its tokens if need_s is 0 or N_s blocks
//   are free, and T_s tokens fit the step's lists;
//   new block i of s = queue[(head + N_s - need_s + i) mod capacity],
//   slot of the token at position p = block(p / bs) * bs + p % bs.
// The sums never decrease, so a granted sequence's blocks start where those of the
// granted ones before it end, and two prefix sums settle everything.
//
// Work split.  Every CTA makes both prefix sums of the whole batch in its shared
// memory (a few loads and shuffles a thread), so that the CTAs need neither each
// other nor a workspace, and fills its share of the token lists and new table
// entries, finding a token's sequence by bisection.  The lengths and the queue's
// state, which may be updated in place, are written by the CTA itself where there
// is one, and else by a launch behind it (one cluster of 8 CTAs that meets before
// it writes took 35 us for 262,144 tokens of 1,000 sequences).  Bound: latency (a
// launch, three dependent rounds of loads); a token costs 12 bytes.  256 tokens of as
// many sequences take 4.2 us in a graph, 262,144 tokens of 1,000 sequences 9.4.
#include <cooperative_groups.h>

#include "device_utils.cuh"

namespace pkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// Inclusive sums of two values over the block; `tmp` holds 2 * kWarps values.
// Every thread gets the block's totals too.
template <class A, class B>
__device__ __forceinline__ void block_scan(A& a, B& b, A& a_all, B& b_all, int64_t* tmp) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const A x = __shfl_up_sync(0xffffffffu, a, o);
        const B y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        tmp[w] = a;
        tmp[kWarps + w] = b;
    }
    __syncthreads();
    if (w == 0) {
        int64_t x = tmp[lane], y = tmp[kWarps + lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
            const int64_t v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x += u;
                y += v;
            }
        }
        tmp[lane] = x;
        tmp[kWarps + lane] = y;
    }
    __syncthreads();
    if (w > 0) {
        a += static_cast<A>(tmp[w - 1]);
        b += static_cast<B>(tmp[kWarps + w - 1]);
    }
    a_all = static_cast<A>(tmp[kWarps - 1]);
    b_all = static_cast<B>(tmp[2 * kWarps - 1]);
    __syncthreads();  // tmp may be written again
}

// Largest s in [0, n) with first[s] <= x (non-decreasing, first[0] = 0).
__device__ __forceinline__ int owner(const int32_t* first, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct Queue {
    int head, count;
    bool sound;  // else it is taken as empty
};

__device__ __forceinline__ Queue queue_of(const int32_t* state, int capacity, uint32_t* status) {
    Queue q{state[0], state[1], true};
    if (q.head < 0 || q.head >= capacity || q.count < 0 || q.count > capacity) {
        if (threadIdx.x == 0) raise_flag(status, kFlagBadQueue);
        q = Queue{0, 0, false};
    }
    return q;
}

// (head + x) mod capacity, 0 <= x <= capacity.
__device__ __forceinline__ int ring(int head, int x, int capacity) {
    const uint32_t y = static_cast<uint32_t>(head) + static_cast<uint32_t>(x);
    return static_cast<int>(y >= static_cast<uint32_t>(capacity) ? y - static_cast<uint32_t>(capacity) : y);
}

// What a launch writes: the lists and table entries, or the lengths and the queue's
// state, or both (one CTA).
enum Part { kBoth, kLists, kLengths };

template <Part kPart>
__global__ void __launch_bounds__(kThreads, 1) kv_tables_extend_kernel(const TablesArgs a) {
    extern __shared__ int32_t lists[];
    __shared__ int64_t tmp[2 * kWarps];
    const int rank = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
    const int B = a.num_seqs, bs = a.block_size, tid = threadIdx.x;
    int32_t* first_token = lists;              // [B] of each sequence, among the step's
    int32_t* first_block = lists + B;          // [B] of each sequence, among the step's new ones
    int32_t* held = lists + 2 * B;             // [B] cached tokens
    pdl_allow_next();
    pdl_wait();
    const bool reports = rank == 0 && kPart != kLengths;
    const Queue q = queue_of(a.queue_state, a.num_blocks, reports ? a.status : nullptr);

    int64_t asked_tokens = 0, asked_blocks = 0;  // of the sequences before these
    int tokens = 0, blocks = 0;                  // granted
    for (int base = 0; base < B; base += kThreads) {
        const int s = base + tid;
        int c = 0, n = 0, need = 0;
        if (s < B) {
            c = a.cached_lens[s];
            n = a.new_lens[s];
            const int64_t end = static_cast<int64_t>(c) + n;
            if (c < 0 || n < 0 || end > static_cast<int64_t>(a.max_blocks) * bs) {
                if (reports) raise_flag(a.status, kFlagBadContext);
                n = 0;
            } else {
                need = static_cast<int>((end + bs - 1) / bs) - (c + bs - 1) / bs;
            }
        }
        int64_t upto_tokens = n, upto_blocks = need, all_tokens, all_blocks;
        block_scan(upto_tokens, upto_blocks, all_tokens, all_blocks, tmp);
        const bool granted = (need == 0 || asked_blocks + upto_blocks <= q.count) &&
                             asked_tokens + upto_tokens <= a.num_tokens;
        if (!granted) n = need = 0;
        asked_tokens += all_tokens;
        asked_blocks += all_blocks;
        int t = n, b = need, t_all, b_all;
        block_scan(t, b, t_all, b_all, tmp);
        if (s < B) {
            first_token[s] = tokens + t - n;
            first_block[s] = blocks + b - need;
            held[s] = c;
        }
        tokens += t_all;
        blocks += b_all;
    }
    __syncthreads();  // the CTA has read what it needs of the buffers that are now written
    if constexpr (kPart != kLists) {
        for (int s = tid; s < B; s += kThreads) {
            const int n = (s + 1 < B ? first_token[s + 1] : tokens) - first_token[s];
            a.query_start[s] = first_token[s];
            a.context_lens[s] = held[s] + n;
        }
        if (tid == 0) {
            a.query_start[B] = tokens;
            a.queue_state_out[0] = ring(q.head, blocks, a.num_blocks);
            a.queue_state_out[1] = q.count - blocks;
        }
    }
    if constexpr (kPart == kLengths) return;
    // New block x of the step, as its table entry (-1: the queue holds no block there).
    auto block_at = [&](int x) {
        const int id = a.free_queue[ring(q.head, x, a.num_blocks)];
        if (id >= 0 && id < a.num_blocks) return id;
        raise_flag(a.status, kFlagBadQueue);
        return -1;
    };
    for (int x = rank * kThreads + tid; x < blocks; x += ctas * kThreads) {
        const int s = owner(first_block, B, x);
        const int j = (held[s] + bs - 1) / bs + x - first_block[s];
        a.block_tables[static_cast<int64_t>(s) * a.max_blocks + j] = block_at(x);
    }
    for (int64_t t = rank * kThreads + tid; t < a.num_tokens; t += ctas * kThreads) {
        int slot = -1, pos = 0, s = -1;
        if (t < tokens) {
            s = owner(first_token, B, static_cast<int>(t));
            const int c = held[s];
            pos = c + static_cast<int>(t) - first_token[s];
            const int j = pos / bs, old = (c + bs - 1) / bs;
            int id;
            if (j < old) {
                id = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + j];
                if (id < 0 || id >= a.num_blocks) {
                    raise_flag(a.status, kFlagBadBlock);
                    id = -1;
                }
            } else {
                id = block_at(first_block[s] + j - old);
            }
            if (id >= 0) slot = id * bs + (pos - j * bs);
        }
        a.slot_mapping[t] = slot;
        a.positions[t] = pos;
        a.seq_ids[t] = s;
    }
}

// Blocks go back in the order of the sequences, each one's in table order: a warp
// counts its row's, the counts are shared through the cluster's shared memory, and
// after their prefix sum the warp writes its row's into the ring.
__global__ void __launch_bounds__(kThreads, 1) kv_tables_release_kernel(const TablesArgs a) {
    extern __shared__ int32_t lists[];
    __shared__ int64_t tmp[2 * kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
    const int B = a.num_seqs, bs = a.block_size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* mine = lists;       // [B] counts of this CTA's rows
    int32_t* first = lists + B;  // [B] place of each row's first block among those given back
    pdl_allow_next();
    pdl_wait();
    const Queue q = queue_of(a.queue_state, a.num_blocks, rank == 0 ? a.status : nullptr);

    // Entries [from, to) of row s whose blocks go back.
    auto range_of = [&](int s, int* from, int* to) {
        int c = a.context_lens[s];
        if (c < 0 || c > static_cast<int64_t>(a.max_blocks) * bs) {
            if (lane == 0) raise_flag(a.status, kFlagBadContext);
            c = 0;
        }
        if (a.finished && a.finished[s] != 0) {
            *from = 0;
            *to = (c + bs - 1) / bs;
            return true;
        }
        // The next query stands at c and sees the positions from c - window + 1 on.
        *from = a.window > 0 ? static_cast<int>((static_cast<int64_t>(a.sinks) + bs - 1) / bs) : 0;
        *to = a.window > 0 && c + 1 > a.window ? (c + 1 - a.window) / bs : 0;
        return false;
    };
    auto held = [&](int s, int e, int to) {
        if (e >= to) return -1;
        const int id = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + e];
        if (id >= a.num_blocks) raise_flag(a.status, kFlagBadBlock);
        return id < a.num_blocks ? id : -1;
    };
    const int step = ctas * kWarps;
    for (int s = warp * ctas + rank; s < B; s += step) {
        int from, to, n = 0;
        range_of(s, &from, &to);
        for (int e = from + lane; e < to; e += 32) n += held(s, e, to) >= 0;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == 0) mine[s] = n;
    }
    cluster.sync();
    int total = 0;
    for (int base = 0; base < B; base += kThreads) {
        const int s = base + tid;
        int n = s < B ? cluster.map_shared_rank(mine, s % ctas)[s] : 0;
        int x = n, y = 0, all, unused;
        block_scan(x, y, all, unused, tmp);
        if (s < B) first[s] = total + x - n;
        total += all;
    }
    cluster.sync();  // counts and queue state are read everywhere
    // No queue, or more blocks than there are: nothing goes back.
    if (!q.sound || static_cast<int64_t>(q.count) + total > a.num_blocks) {
        if (rank == 0 && tid == 0) raise_flag(a.status, kFlagBadQueue);
        return;
    }
    const int tail = ring(q.head, q.count, a.num_blocks);
    for (int s = warp * ctas + rank; s < B; s += step) {
        int from, to, at = first[s];
        const bool done = range_of(s, &from, &to);
        for (int e0 = from; e0 < to; e0 += 32) {
            const int id = held(s, e0 + lane, to);
            const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
            if (id >= 0) {
                a.free_queue_out[ring(tail, at + __popc(have & ((1u << lane) - 1u)), a.num_blocks)] = id;
                a.block_tables[static_cast<int64_t>(s) * a.max_blocks + e0 + lane] = -1;
            }
            at += __popc(have);
        }
        __syncwarp();
        if (done && lane == 0) a.context_lens[s] = 0;
    }
    if (rank == 0 && tid == 0) a.queue_state_out[1] = q.count + total;
}

cudaError_t launch_cluster(void (*kernel)(const TablesArgs), RaisedLimit* limit, const TablesArgs& a, int smem, int ctas,
                           cudaStream_t stream) {
    const cudaError_t e = allow_shared_memory(kernel, a.device, smem, limit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_tables_extend(const TablesArgs& a, int num_sms, cudaStream_t stream) {
    static RaisedLimit limits[3];
    const int smem = 3 * 4 * a.num_seqs;
    auto launch = [&](auto kernel, RaisedLimit* limit, int ctas) {
        const cudaError_t e = allow_shared_memory(kernel, a.device, smem, limit);
        if (e != cudaSuccess) return e;
        return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), static_cast<size_t>(smem), stream, true, a);
    };
    // One CTA while a thread has four tokens at most; else two tokens a thread, on one CTA an SM at most.
    const int64_t ctas = (static_cast<int64_t>(a.num_tokens) + 2 * kThreads - 1) / (2 * kThreads);
    if (ctas <= 2) return launch(kv_tables_extend_kernel<kBoth>, &limits[0], 1);
    const cudaError_t e = launch(kv_tables_extend_kernel<kLists>, &limits[1], static_cast<int>(ctas < num_sms ? ctas : num_sms));
    if (e != cudaSuccess) return e;
    return launch(kv_tables_extend_kernel<kLengths>, &limits[2], 1);
}

cudaError_t launch_tables_release(const TablesArgs& a, cudaStream_t stream) {
    static RaisedLimit limit;
    int ctas = 1;  // one while a warp has one row
    while (ctas < kMaxCluster && a.num_seqs > kWarps * ctas) ctas <<= 1;
    return launch_cluster(kv_tables_release_kernel, &limit, a, 2 * 4 * a.num_seqs, ctas, stream);
}

}  // namespace pkv
