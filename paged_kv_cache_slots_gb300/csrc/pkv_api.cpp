// C ABI of the paged KV cache library: validation, pool bookkeeping, launch
// planning, tensor-map encoding and status handling.  Every argument is
// checked here, before anything reaches the device.
#include "pkv.h"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <deque>
#include <mutex>
#include <new>
#include <unordered_map>
#include <vector>

#include "pkv_internal.h"
#include "shared_prefix.cuh"

using namespace pkv;

namespace {

thread_local char g_last_error[512] = "";

kv_status_t fail(kv_status_t st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return st;
}

kv_status_t cuda_fail(cudaError_t e, const char* what) {
    return fail(KV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool valid_dtype(int d) { return d == KV_F32 || d == KV_F16 || d == KV_BF16; }
bool valid_pool_dtype(int d) { return valid_dtype(d) || d == KV_FP8_E4M3; }
bool valid_scale(float x) { return std::isfinite(x) && x > 0.f; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Restores the caller's current device on scope exit.
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) return;
        ok = (prev == dev) || (cudaSetDevice(dev) == cudaSuccess);
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

constexpr int kMaxDevices = 64;
std::mutex g_dev_mutex;
uint32_t* g_status_ptr[kMaxDevices] = {};
int g_sm_count[kMaxDevices] = {};
int g_max_smem[kMaxDevices] = {};
int g_smem_per_sm[kMaxDevices] = {};

// Per-device facts and the status word of the current device.
kv_status_t device_info(int* dev_out, uint32_t** status, int* sms, int* max_smem, int* smem_sm) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(KV_ERR_UNSUPPORTED, "device ordinal %d", dev);
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (g_status_ptr[dev] == nullptr) {
        int v = 0;
        if ((e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
        g_sm_count[dev] = v;
        g_max_smem[dev] = max_dynamic_smem(dev);
        if ((e = cudaDeviceGetAttribute(&v, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev)) !=
            cudaSuccess)
            return cuda_fail(e, "cudaDeviceGetAttribute(shared memory per SM)");
        g_smem_per_sm[dev] = v;
        uint32_t* p = nullptr;
        if ((e = status_word_address(&p)) != cudaSuccess) return cuda_fail(e, "status word address");
        g_status_ptr[dev] = p;
    }
    if (dev_out) *dev_out = dev;
    if (status) *status = g_status_ptr[dev];
    if (sms) *sms = g_sm_count[dev];
    if (max_smem) *max_smem = g_max_smem[dev];
    if (smem_sm) *smem_sm = g_smem_per_sm[dev];
    return KV_OK;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Options {
    int num_ctas, ctas_per_sm, consumer_warps, kernel, heads_per_stage, separate_reduce, no_pdl,
        early_reads, test_stall;
};

kv_status_t read_options(const kv_decode_options_t* o, Options* out) {
    Options r{0, 1, 0, KV_KERNEL_AUTO, 0, 0, 0, 0, 0};
    if (o) {
        if (o->num_ctas < 0 || o->ctas_per_sm < 0 || o->consumer_warps < 0 ||
            o->consumer_warps > 15 || o->ctas_per_sm > 8 || o->heads_per_stage < 0 ||
            o->heads_per_stage > 15)
            return fail(KV_ERR_INVALID_ARG, "decode options out of range");
        if (o->kernel != KV_KERNEL_AUTO && o->kernel != KV_KERNEL_FFMA && o->kernel != KV_KERNEL_MMA)
            return fail(KV_ERR_INVALID_ARG, "unknown kernel selector %d", static_cast<int>(o->kernel));
        if (o->num_ctas) r.num_ctas = o->num_ctas;
        if (o->ctas_per_sm) r.ctas_per_sm = o->ctas_per_sm;
        r.consumer_warps = o->consumer_warps;
        r.kernel = o->kernel;
        r.heads_per_stage = o->heads_per_stage;
        r.separate_reduce = o->separate_reduce != 0;
        r.no_pdl = o->no_pdl != 0;
        r.early_reads = o->early_reads != 0;
        r.test_stall = o->test_stall != 0;
    }
    *out = r;
    return KV_OK;
}

int grid_size(const Options& o, int sms) { return o.num_ctas > 0 ? o.num_ctas : sms * o.ctas_per_sm; }

// Workspace layout: counters [B*Hkv] int32 (must be zero between calls),
// partial O, partial (max, sum), per-sequence prefix [B+1].  The partial
// areas are sized for any head chunking: slots * Hc <= (P + B) * Hkv.
struct WsLayout {
    size_t counters, part_o, part_ml, cum, total;
};

WsLayout workspace_layout(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int ctas) {
    WsLayout w;
    const size_t rows = (static_cast<size_t>(ctas) + num_seqs) * num_q_heads;  // (P + B) * Hkv * G
    w.counters = 0;
    w.part_o = align256(static_cast<size_t>(num_seqs) * num_kv_heads * 4);
    w.part_ml = w.part_o + align256(rows * head_dim * 4);
    w.cum = w.part_ml + align256(rows * 2 * 4);
    w.total = w.cum + align256(static_cast<size_t>(num_seqs + 1) * 4);
    return w;
}

// KV heads per pipeline stage: the largest divisor of Hkv whose K slab of one
// block fits 32 KiB (and, for the tensor copies, 256 box rows).
int auto_heads_per_stage(int num_kv_heads, int block_size, int head_dim, int dtype, bool tensor) {
    const int head_bytes = block_size * head_dim * dtype_bytes(dtype);
    for (int hc = num_kv_heads < 15 ? num_kv_heads : 15; hc > 1; --hc) {
        if (num_kv_heads % hc) continue;
        if (hc * head_bytes > 32768) continue;
        if (tensor && hc * block_size > 256) continue;
        return hc;
    }
    return 1;
}

// Stages for *R warps per head, or for fewer where the ring would hold less
// than two stages per replica (each replica owns every R-th stage).  keep_warps:
// an explicit warp count is kept if it fits at all.
bool plan_warps(int kernel, int kv_dtype, int head_dim, int block_size, int G, int num_seqs, int hc, int budget,
                bool keep_warps, int* R, DecodePlan* plan) {
    bool planned = false;
    for (; *R >= 1; --*R) {
        planned = decode_plan(kernel, kv_dtype, head_dim, block_size, G, num_seqs, hc, *R, budget, plan);
        if (planned && (plan->stages >= 2 * *R || *R == 1)) break;
        if (planned && keep_warps) break;
    }
    return planned;
}

// Phantom items per pair: about the time a CTA loses switching to the
// next pair (the partial's stores, the merge arrival's release fence,
// the next q: 3-5 us measured) in stages' worth of streaming, i.e.
// 300 KiB of stage data: 5 items for 64 KiB stages, 8 (the cap) for the
// E4M3 stages of 32 KiB (the best of 0, 100, 200, 300 and 400 KiB in an
// A/B on one box).  Not with too few items to split (fewer than two a
// CTA even with every table entry used).
int phantom_items(int num_seqs, int chunks, int max_blocks, int ctas, int stage_half_bytes) {
    const int64_t stage_bytes = 2 * static_cast<int64_t>(stage_half_bytes);
    const int64_t max_items = static_cast<int64_t>(num_seqs) * chunks * max_blocks;
    const int ph = static_cast<int>((int64_t{300} * 1024 + stage_bytes / 2) / stage_bytes);
    return max_items >= 2 * static_cast<int64_t>(ctas) ? (ph > 8 ? 8 : ph) : 0;
}

// What a windowed query sees: see paged_window_decode_attention.
struct Sight {
    int window, sinks;
};

// Whether a windowed decode takes the kernel for small calls (window_decode_small.cu) rather than the persistent
// one: by estimates of both kernels' times with every sequence as long as its window.  From 892 calls measured with
// either kernel (graphs, inputs out of L2; 1, 2 and 8 KV heads, windows of 128 to 131,072, batches of 1 to 256):
//   Small: a wave of CTAs takes 6 us and, for each block that its warps take one after the other, 0.3 us and 0.16 a KiB
//   of the block's K rows (0.21 over E4M3; 0.65 of it where three warps or fewer share an SM's shared memory); all of
//   them no less than 4.5 TB/s allow (5 with blocks from 16 KiB on, 5.5 with smaller ones and one wave; over E4M3 0.92 of
//   that).  Of 8-CTA clusters three quarters fit at once (16 pairs: 70 us, 4 pairs: 33).
//   Persistent: 15 us and the rate that its stages reach: blocks of few heads make small stages (64 sequences, one KV head of
//   128, blocks of 16, window 8,192: 126 us, small 53), blocks of 24 KiB a head leave it two (16 sequences, 8 KV heads,
//   blocks of 128, window 8,192: 188, small 107); one long sequence is cut into so many parts that the merge takes 60.
// The small kernel gives a sequence of any length the same CTAs, and lengths are not known here: one long sequence
// among short ones waits for its own CTAs alone, where the persistent kernel spreads it over every SM (window 32,768,
// 1 of 32, 8 KV heads, blocks of 64: 237 us, persistent 47).  So what a CTA may have to stream is bounded: 1.1 MB,
// or 4.4 MB where the persistent kernel would take a quarter longer on equal lengths.  Of the measured calls some 55 are more
// than 10 % above the faster kernel: lengths far apart (up to 2.6x), and what that bound costs equal ones.
bool small_window(const SmallPlan& plan, int num_seqs, int kv_heads, int row_blocks, int half, bool fp8, int sms) {
    const double bytes = 2.0 * half * row_blocks * num_seqs * kv_heads, h = half / 1024.0;
    const double fit = static_cast<double>(sms) * plan.per_sm * (plan.ctas == 8 ? 0.75 : 1.0);
    double waves = static_cast<double>(num_seqs) * kv_heads * plan.ctas / fit;
    waves = waves < 1 ? 1 : waves < 3 ? std::ceil(waves) : waves;
    const double step = 0.3 + h * (fp8 ? 0.21 : 0.16) * (plan.warps <= 3 ? 0.65 : 1.0);
    const int chain = (row_blocks + plan.ctas * plan.warps - 1) / (plan.ctas * plan.warps);
    double small = waves * (6 + chain * step);  // us
    const double stream = 5 + bytes / ((h >= 16 ? 5.0e6 : waves > 1 ? 4.5e6 : 5.5e6) * (fp8 ? 0.92 : 1.0));
    if (small < stream) small = stream;
    double rate;  // GB/s
    if (h >= 24)
        rate = 2900;
    else if (h >= 16)
        rate = fp8 ? (kv_heads > 1 ? 3400 : 4700) : (kv_heads > 1 ? 4700 : 6000);
    else
        rate = h * kv_heads < 8 ? 2300 : h * kv_heads < 16 ? 4200 : h * kv_heads < 32 ? 5500 : 6300;
    double persistent = 15 + bytes / rate / 1000;
    if (num_seqs == 1 && bytes > 4e6 && persistent < 60) persistent = 60;
    const double kib = 2 * h * row_blocks / plan.ctas;
    return small < persistent && (kib <= 1100 || (kib <= 4400 && 1.25 * small < persistent));
}

kv_status_t check_sight(const Sight& w, int max_blocks, int block_size) {
    if (w.window < 1 || w.sinks < 0)
        return fail(KV_ERR_INVALID_ARG, "window %d (from 1 on), sinks %d (from 0 on)", w.window, w.sinks);
    if (static_cast<int64_t>(max_blocks) * block_size >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "a table row of more than 2^31 tokens");
    return KV_OK;
}

// The same in a kernel's arguments, each no larger than a table row.
template <class Args>
void set_sight(const Sight& w, int max_blocks, int block_size, Args* a) {
    const int cap = max_blocks * block_size;
    a->window = w.window < cap ? w.window : cap;
    a->sinks = w.sinks < cap ? w.sinks : cap;
    a->sink_blocks = (a->sinks + block_size - 1) / block_size;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 2-D view of one layer's cache: rows = num_blocks*Hkv*bs, row = head_dim
// elements; box = 128 bytes (64 f16/bf16 or 128 E4M3 elements) x box_rows
// rows (Hc heads of one block), 128-byte swizzle.
kv_status_t encode_cache_map(CUtensorMap* map, const void* base, int dtype, int rows, int head_dim,
                             int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return fail(KV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const int eb = dtype_bytes(dtype);
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_dim) * eb};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / eb), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1u, 1u};
    const CUtensorMapDataType type = dtype == KV_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : dtype == KV_F16  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    CUresult r = enc(map, type,
                     2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(KV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return KV_OK;
}

// 4-D view of one layer's cache for the windowed prefill: 64 elements, 8 rows, the
// row's 64-element slices, groups of 8 rows; box = `box_rows` rows with all slices,
// 128-byte swizzle, so that a box lands group by group, slice by slice within one.
kv_status_t encode_group_map(CUtensorMap* map, const void* base, int dtype, int rows, int head_dim, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return fail(KV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t row = static_cast<cuuint64_t>(head_dim) * 2;
    cuuint64_t dims[4] = {64, 8, static_cast<cuuint64_t>(head_dim / 64), static_cast<cuuint64_t>(rows / 8)};
    cuuint64_t strides[3] = {row, 128, 8 * row};
    cuuint32_t box[4] = {64u, 8u, static_cast<cuuint32_t>(head_dim / 64), static_cast<cuuint32_t>(box_rows / 8)};
    cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    CUresult r = enc(map, dtype == KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                     const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(KV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return KV_OK;
}

// 3-D view of the query rows [tokens][heads][head_dim]; box = 64 elements x
// box_heads x box_tokens, 128-byte swizzle.
kv_status_t encode_query_map(CUtensorMap* map, const void* q, int dtype, int tokens, int heads, int head_dim,
                             int box_heads, int box_tokens) {
    auto enc = tensor_map_encoder();
    if (!enc) return fail(KV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t row = static_cast<cuuint64_t>(head_dim) * 2;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    cuuint64_t strides[2] = {row, row * heads};
    cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    CUresult r = enc(map, dtype == KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                     const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(KV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return KV_OK;
}

}  // namespace

kv_status_t pkv::report_error(kv_status_t st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return st;
}

// ------------------------------------------------------------------ pool
struct kv_pool {
    kv_pool_config_t cfg;
    char* base;
    bool owned;
    size_t layer_bytes;  // one of K or V for one layer
    kv_block_allocator_t* alloc = nullptr;  // kv_seq_extend / kv_seq_free, created on first use
};

// ------------------------------------------------------------------ rope
struct kv_rope {
    int rot_dim, interleaved, num_axes;
    float amplitude;
    uint64_t phase[kMaxRopePairs];
    uint8_t axis[kMaxRopePairs];
};

namespace {

// f / (2 pi) turns, modulo 1, as 64-bit fixed point.  1 / (2 pi) is taken as
// a double and what that leaves, and the product's own rounding error from an
// fma: for |f| up to 2^20 the result is the nearest multiple of 2^-64, or its
// neighbour.
uint64_t turns_fixed_point(double f) {
    constexpr double kInv2Pi = 0.15915494309189535, kInv2PiRest = -9.839338337591243e-18;
    const double hi = f * kInv2Pi;
    const double lo = std::fma(f, kInv2Pi, -hi) + f * kInv2PiRest;
    auto fixed = [](double x) {
        double t = std::ldexp(x - std::rint(x), 64);  // x - rint(x) is exact
        if (t >= 0x1p63) t -= 0x1p64;
        return static_cast<uint64_t>(static_cast<int64_t>(std::rint(t)));
    };
    return fixed(hi) + fixed(lo);
}

// Whether rows of `row` bytes, `n` of them `stride` bytes apart, at p and at o
// can touch one another.
bool rows_overlap(const void* p, int64_t p_stride, int64_t p_row, const void* o, int64_t o_stride,
                  int64_t o_row, int64_t n) {
    const int64_t a = reinterpret_cast<intptr_t>(p), b = reinterpret_cast<intptr_t>(o);
    const int64_t a_end = a + (n - 1) * p_stride + p_row, b_end = b + (n - 1) * o_stride + o_row;
    if (a_end <= b || b_end <= a) return false;
    // Slices of one packed buffer: apart inside every row of it.
    if (n > 1 && p_stride == o_stride) {
        int64_t d = (b - a) % p_stride;
        if (d < 0) d += p_stride;
        return d < p_row || p_stride - d < o_row;
    }
    return true;
}

// Whether `bytes` bytes at p touch one of `n` rows of `row` bytes, `stride` apart, at o.
bool touches_rows(const void* p, int64_t bytes, const void* o, int64_t stride, int64_t row, int64_t n) {
    const int64_t a = reinterpret_cast<intptr_t>(p), b = reinterpret_cast<intptr_t>(o);
    if (a + bytes <= b || b + (n - 1) * stride + row <= a) return false;
    const int64_t d = a - b;
    return d < 0 || d % stride < row || d % stride + bytes > stride;
}

}  // namespace

// ---------------------------------------------------------------- allocator
struct kv_block_allocator {
    int num_blocks = 0, block_size = 0;
    std::deque<int32_t> free_q;
    struct Seq {
        std::vector<int32_t> table;
        int64_t tokens = 0;
    };
    std::unordered_map<int64_t, Seq> seqs;
};

namespace {

// Moves blocks between the pool and a buffer the GPU can address.
kv_status_t swap_blocks(kv_pool_t* p, const int32_t* block_ids, int n, void* host,
                        size_t host_bytes, bool to_host, void* stream) {
    const char* what = to_host ? "kv_swap_out" : "kv_swap_in";
    if (!p) return fail(KV_ERR_INVALID_ARG, "%s: null pool", what);
    if (n < 0) return fail(KV_ERR_INVALID_ARG, "%s: %d blocks", what, n);
    if (n == 0) return KV_OK;
    if (!block_ids || !host) return fail(KV_ERR_INVALID_ARG, "%s: null pointer", what);
    const size_t need = kv_swap_bytes(p, n);
    if (host_bytes < need)
        return fail(KV_ERR_INVALID_ARG, "%s: host buffer of %zu bytes < %zu needed", what,
                    host_bytes, need);
    if (!aligned(host, 16)) return fail(KV_ERR_INVALID_ARG, "%s: host buffer must be 16-byte aligned", what);
    DeviceGuard g(p->cfg.device);
    if (!g.ok) return fail(KV_ERR_CUDA, "cannot select device %d", p->cfg.device);
    // The kernel dereferences both pointers: they must be memory the GPU
    // addresses (page-locked or registered host memory, managed or device
    // memory), not plain pageable memory.
    void* dev_ptrs[2] = {host, const_cast<int32_t*>(block_ids)};
    for (int k = 0; k < 2; ++k) {
        cudaPointerAttributes attr{};
        cudaError_t e = cudaPointerGetAttributes(&attr, dev_ptrs[k]);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return cuda_fail(e, "cudaPointerGetAttributes");
        }
        if (attr.type == cudaMemoryTypeUnregistered)
            return fail(KV_ERR_INVALID_ARG,
                        "%s: %s is pageable host memory; use page-locked (cudaHostAlloc / "
                        "cudaHostRegister), managed or device memory", what,
                        k == 0 ? "the host buffer" : "block_ids");
        if (attr.type == cudaMemoryTypeHost) {
            if (!attr.devicePointer)
                return fail(KV_ERR_INVALID_ARG, "%s: host memory not mapped for the device", what);
            dev_ptrs[k] = attr.devicePointer;
        }
    }
    uint32_t* status = nullptr;
    int sms = 0;
    if (kv_status_t st = device_info(nullptr, &status, &sms, nullptr, nullptr)) return st;
    SwapArgs a{p->base,
               static_cast<char*>(dev_ptrs[0]),
               static_cast<const int32_t*>(dev_ptrs[1]),
               status,
               static_cast<int64_t>(p->layer_bytes),
               static_cast<int64_t>(p->layer_bytes / p->cfg.num_blocks),
               n,
               p->cfg.num_layers,
               p->cfg.num_blocks,
               to_host ? 1 : 0,
               1};
    cudaError_t e = launch_swap(a, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "swap launch");
    return KV_OK;
}

}  // namespace

extern "C" {

const char* kv_status_string(kv_status_t s) {
    switch (s) {
        case KV_OK: return "KV_OK";
        case KV_ERR_INVALID_ARG: return "KV_ERR_INVALID_ARG";
        case KV_ERR_UNSUPPORTED: return "KV_ERR_UNSUPPORTED";
        case KV_ERR_OUT_OF_MEMORY: return "KV_ERR_OUT_OF_MEMORY";
        case KV_ERR_OUT_OF_BLOCKS: return "KV_ERR_OUT_OF_BLOCKS";
        case KV_ERR_WORKSPACE_TOO_SMALL: return "KV_ERR_WORKSPACE_TOO_SMALL";
        case KV_ERR_CUDA: return "KV_ERR_CUDA";
        case KV_ERR_DEVICE_CHECK: return "KV_ERR_DEVICE_CHECK";
        case KV_ERR_DEVICE_TIMEOUT: return "KV_ERR_DEVICE_TIMEOUT";
        case KV_ERR_NOT_FOUND: return "KV_ERR_NOT_FOUND";
    }
    return "KV_ERR_UNKNOWN";
}

const char* kv_last_error(void) { return g_last_error; }

size_t kv_pool_bytes(const kv_pool_config_t* c) {
    if (!c || c->num_layers <= 0 || c->num_blocks <= 0 || c->block_size <= 0 || c->num_kv_heads <= 0 ||
        c->head_dim <= 0 || !valid_pool_dtype(c->dtype))
        return 0;
    return 2ull * c->num_layers * c->num_blocks * c->block_size * c->num_kv_heads * c->head_dim *
           static_cast<size_t>(dtype_bytes(c->dtype));
}

kv_status_t kv_pool_create(const kv_pool_config_t* cfg, void* buffer, size_t buffer_bytes,
                           kv_pool_t** out) {
    if (!cfg || !out) return fail(KV_ERR_INVALID_ARG, "kv_pool_create: null argument");
    *out = nullptr;
    const size_t bytes = kv_pool_bytes(cfg);
    if (bytes == 0) return fail(KV_ERR_INVALID_ARG, "kv_pool_create: invalid configuration");
    if (cfg->block_size > 1024) return fail(KV_ERR_INVALID_ARG, "block_size %d > 1024", cfg->block_size);
    if ((static_cast<size_t>(cfg->head_dim) * dtype_bytes(cfg->dtype)) % 16)
        return fail(KV_ERR_INVALID_ARG, "head_dim * element size must be a multiple of 16 bytes");
    if (static_cast<int64_t>(cfg->num_blocks) * cfg->block_size >= (int64_t{1} << 31) ||
        static_cast<int64_t>(cfg->num_blocks) * cfg->block_size * cfg->num_kv_heads >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "pool too large for 32-bit slot / row indices");
    if (cfg->device < 0) return fail(KV_ERR_INVALID_ARG, "device %d", cfg->device);
    if (buffer) {
        if (buffer_bytes < bytes)
            return fail(KV_ERR_INVALID_ARG, "buffer of %zu bytes < %zu needed", buffer_bytes, bytes);
        if (!aligned(buffer, 256)) return fail(KV_ERR_INVALID_ARG, "pool buffer must be 256-byte aligned");
    }
    kv_pool* p = new (std::nothrow) kv_pool;
    if (!p) return fail(KV_ERR_OUT_OF_MEMORY, "host allocation failed");
    p->cfg = *cfg;
    p->layer_bytes = bytes / (2ull * cfg->num_layers);
    p->owned = buffer == nullptr;
    p->base = static_cast<char*>(buffer);
    if (!buffer) {
        DeviceGuard g(cfg->device);
        if (!g.ok) {
            delete p;
            return fail(KV_ERR_CUDA, "cannot select device %d", cfg->device);
        }
        void* mem = nullptr;
        cudaError_t e = cudaMalloc(&mem, bytes);
        if (e != cudaSuccess) {
            delete p;
            cudaGetLastError();
            return fail(KV_ERR_OUT_OF_MEMORY, "cudaMalloc(%zu): %s", bytes, cudaGetErrorString(e));
        }
        p->base = static_cast<char*>(mem);
    }
    *out = p;
    return KV_OK;
}

void kv_pool_destroy(kv_pool_t* p) {
    if (!p) return;
    if (p->owned && p->base) {
        DeviceGuard g(p->cfg.device);
        cudaFree(p->base);
    }
    kv_allocator_destroy(p->alloc);
    delete p;
}

kv_status_t kv_pool_layer(const kv_pool_t* p, int layer, void** k, void** v) {
    if (!p || !k || !v) return fail(KV_ERR_INVALID_ARG, "kv_pool_layer: null argument");
    if (layer < 0 || layer >= p->cfg.num_layers)
        return fail(KV_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, p->cfg.num_layers);
    *k = p->base + (2ull * layer) * p->layer_bytes;
    *v = p->base + (2ull * layer + 1) * p->layer_bytes;
    return KV_OK;
}

kv_status_t kv_pool_config(const kv_pool_t* p, kv_pool_config_t* c) {
    if (!p || !c) return fail(KV_ERR_INVALID_ARG, "kv_pool_config: null argument");
    *c = p->cfg;
    return KV_OK;
}

kv_status_t kv_slot_mapping(const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                            int num_seqs, int block_size, int num_blocks, int32_t* slot_mapping,
                            void* stream) {
    if (num_seqs < 0 || max_blocks <= 0 || block_size <= 0 || num_blocks <= 0)
        return fail(KV_ERR_INVALID_ARG, "kv_slot_mapping: sizes out of range");
    if (num_seqs == 0) return KV_OK;
    if (!block_tables || !context_lens || !slot_mapping)
        return fail(KV_ERR_INVALID_ARG, "kv_slot_mapping: null pointer");
    if (static_cast<int64_t>(num_blocks) * block_size >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "slots do not fit in int32");
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(nullptr, &status, nullptr, nullptr, nullptr)) return st;
    SlotArgs a{block_tables, context_lens, slot_mapping, status, max_blocks, num_seqs, block_size, num_blocks,
               1};
    cudaError_t e = launch_slot_mapping(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "slot mapping launch");
    return KV_OK;
}

kv_status_t kv_append(kv_pool_t* p, int layer, const int32_t* seq_ids, int n_tokens, const void* k,
                      const void* v, const int32_t* slot_mapping, void* stream) {
    if (!p) return fail(KV_ERR_INVALID_ARG, "kv_append: null pool");
    if (n_tokens < 0) return fail(KV_ERR_INVALID_ARG, "kv_append: n_tokens %d", n_tokens);
    if (p->cfg.dtype == KV_FP8_E4M3)
        return fail(KV_ERR_INVALID_ARG, "kv_append: an E4M3 pool takes kv_append_fp8 (with scales)");
    void *kc = nullptr, *vc = nullptr;
    if (kv_status_t st = kv_pool_layer(p, layer, &kc, &vc)) return st;
    if (n_tokens == 0) return KV_OK;
    if (!k || !v || !slot_mapping) return fail(KV_ERR_INVALID_ARG, "kv_append: null pointer");
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(KV_ERR_INVALID_ARG, "kv_append: k and v must be 16-byte aligned");
    if (static_cast<int64_t>(n_tokens) * p->cfg.num_kv_heads >= (int64_t{1} << 31) / 32)
        return fail(KV_ERR_UNSUPPORTED, "kv_append: too many tokens in one call");
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(nullptr, &status, nullptr, nullptr, nullptr)) return st;
    AppendArgs a{seq_ids, k, v, slot_mapping, kc, vc, status, n_tokens, p->cfg.num_kv_heads,
                 p->cfg.head_dim, p->cfg.block_size, p->cfg.num_blocks, dtype_bytes(p->cfg.dtype), 1,
                 0, p->cfg.dtype, 1.f, 1.f};
    cudaError_t e = launch_append(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
    return KV_OK;
}

kv_status_t kv_append_fp8(kv_pool_t* p, int layer, const int32_t* seq_ids, int n_tokens, const void* k,
                          const void* v, kv_dtype_t src_dtype, const int32_t* slot_mapping, float k_scale,
                          float v_scale, void* stream) {
    if (!p) return fail(KV_ERR_INVALID_ARG, "kv_append_fp8: null pool");
    if (p->cfg.dtype != KV_FP8_E4M3)
        return fail(KV_ERR_INVALID_ARG, "kv_append_fp8: the pool is not KV_FP8_E4M3");
    if (!valid_dtype(src_dtype)) return fail(KV_ERR_INVALID_ARG, "kv_append_fp8: source dtype %d", src_dtype);
    if (!valid_scale(k_scale) || !valid_scale(v_scale))
        return fail(KV_ERR_INVALID_ARG, "kv_append_fp8: scales must be finite and > 0");
    if (n_tokens < 0) return fail(KV_ERR_INVALID_ARG, "kv_append_fp8: n_tokens %d", n_tokens);
    if (p->cfg.head_dim % 16)
        return fail(KV_ERR_UNSUPPORTED, "kv_append_fp8: head_dim must be a multiple of 16");
    void *kc = nullptr, *vc = nullptr;
    if (kv_status_t st = kv_pool_layer(p, layer, &kc, &vc)) return st;
    if (n_tokens == 0) return KV_OK;
    if (!k || !v || !slot_mapping) return fail(KV_ERR_INVALID_ARG, "kv_append_fp8: null pointer");
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(KV_ERR_INVALID_ARG, "kv_append_fp8: k and v must be 16-byte aligned");
    if (static_cast<int64_t>(n_tokens) * p->cfg.num_kv_heads >= (int64_t{1} << 31) / 32)
        return fail(KV_ERR_UNSUPPORTED, "kv_append_fp8: too many tokens in one call");
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(nullptr, &status, nullptr, nullptr, nullptr)) return st;
    AppendArgs a{seq_ids, k, v, slot_mapping, kc, vc, status, n_tokens, p->cfg.num_kv_heads,
                 p->cfg.head_dim, p->cfg.block_size, p->cfg.num_blocks, 1, 1,
                 1, src_dtype, k_scale, v_scale};
    cudaError_t e = launch_append(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
    return KV_OK;
}

kv_status_t kv_rope_create(const kv_rope_config_t* c, kv_rope_t** out) {
    if (!c || !out) return fail(KV_ERR_INVALID_ARG, "kv_rope_create: null argument");
    *out = nullptr;
    if (c->rot_dim < 2 || c->rot_dim % 2)
        return fail(KV_ERR_INVALID_ARG, "kv_rope_create: rot_dim %d is not an even number from 2", c->rot_dim);
    if (c->rot_dim > 2 * kMaxRopePairs)
        return fail(KV_ERR_UNSUPPORTED, "kv_rope_create: rot_dim %d > %d", c->rot_dim, 2 * kMaxRopePairs);
    if (c->num_axes < 1 || c->num_axes > 8)
        return fail(KV_ERR_INVALID_ARG, "kv_rope_create: %d axes (1 .. 8)", c->num_axes);
    if (!std::isfinite(c->amplitude)) return fail(KV_ERR_INVALID_ARG, "kv_rope_create: amplitude is not finite");
    if (!c->inv_freq) return fail(KV_ERR_INVALID_ARG, "kv_rope_create: null inv_freq");
    const int n = c->rot_dim / 2;
    for (int i = 0; i < n; ++i) {
        if (!std::isfinite(c->inv_freq[i])) return fail(KV_ERR_INVALID_ARG, "kv_rope_create: inv_freq[%d] is not finite", i);
        if (c->axis && (c->axis[i] < 0 || c->axis[i] >= c->num_axes))
            return fail(KV_ERR_INVALID_ARG, "kv_rope_create: axis[%d] = %d of %d axes", i, c->axis[i], c->num_axes);
    }
    kv_rope* r = new (std::nothrow) kv_rope;
    if (!r) return fail(KV_ERR_OUT_OF_MEMORY, "host allocation failed");
    memset(r, 0, sizeof *r);
    r->rot_dim = c->rot_dim;
    r->interleaved = c->interleaved != 0;
    r->num_axes = c->num_axes;
    r->amplitude = c->amplitude;
    for (int i = 0; i < n; ++i) {
        r->phase[i] = turns_fixed_point(c->inv_freq[i]);
        r->axis[i] = static_cast<uint8_t>(c->axis ? c->axis[i] : 0);
    }
    *out = r;
    return KV_OK;
}

void kv_rope_destroy(kv_rope_t* r) { delete r; }

// The checks and arguments that kv_append_rope and kv_append_norm_rope (`what`)
// share.  *align: the largest power of two that divides the address of every
// token's rows.  n_tokens 0: nothing but the first checks, *a stays as it is.
static kv_status_t rope_args(const char* what, kv_pool_t* p, int layer, const kv_rope_t* rope, const int32_t* seq_ids,
                             int n_tokens, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             kv_dtype_t src_dtype, const int32_t* slot_mapping, const int32_t* positions,
                             int64_t positions_stride, const void* q, int64_t q_stride, void* q_out,
                             int64_t q_out_stride, int num_q_heads, float k_scale, float v_scale, RopeArgs* a,
                             int* align) {
    if (!p || !rope) return fail(KV_ERR_INVALID_ARG, "%s: null pool or rope", what);
    if (n_tokens < 0) return fail(KV_ERR_INVALID_ARG, "%s: n_tokens %d", what, n_tokens);
    const int D = p->cfg.head_dim, Hkv = p->cfg.num_kv_heads;
    const bool quant = p->cfg.dtype == KV_FP8_E4M3;
    if (!valid_dtype(src_dtype)) return fail(KV_ERR_INVALID_ARG, "%s: source dtype %d", what, src_dtype);
    if (!quant && src_dtype != p->cfg.dtype)
        return fail(KV_ERR_INVALID_ARG, "%s: rows must have the pool's dtype (or the pool be E4M3)", what);
    if (quant && (!valid_scale(k_scale) || !valid_scale(v_scale)))
        return fail(KV_ERR_INVALID_ARG, "%s: scales must be finite and > 0", what);
    if (rope->rot_dim > D)
        return fail(KV_ERR_INVALID_ARG, "%s: rot_dim %d > head_dim %d", what, rope->rot_dim, D);
    void *kc = nullptr, *vc = nullptr;
    if (kv_status_t st = kv_pool_layer(p, layer, &kc, &vc)) return st;
    if (!q) num_q_heads = 0;
    if (num_q_heads < 0 || (q && num_q_heads == 0))
        return fail(KV_ERR_INVALID_ARG, "%s: %d query heads", what, num_q_heads);
    if (n_tokens == 0) return KV_OK;
    if (!k || !v || !slot_mapping || !positions || (q && !q_out))
        return fail(KV_ERR_INVALID_ARG, "%s: null pointer", what);
    const int eb = dtype_bytes(src_dtype);
    const int64_t krow = static_cast<int64_t>(Hkv) * D, qrow = static_cast<int64_t>(num_q_heads) * D;
    if (krow >= (int64_t{1} << 31) || qrow >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "%s: more than 2^31 elements a token", what);
    if (n_tokens > 1 && (k_stride < krow || v_stride < krow || (q && (q_stride < qrow || q_out_stride < qrow))))
        return fail(KV_ERR_INVALID_ARG, "%s: a stride is shorter than a token's rows", what);
    if (rope->num_axes > 1 && positions_stride != 0 && positions_stride < n_tokens)
        return fail(KV_ERR_INVALID_ARG, "%s: positions_stride %lld (0, or from %d tokens on)", what,
                    static_cast<long long>(positions_stride), n_tokens);
    if (!aligned(k, eb) || !aligned(v, eb) || (q && (!aligned(q, eb) || !aligned(q_out, eb))) ||
        !aligned(slot_mapping, 4) || !aligned(positions, 4) || !aligned(seq_ids, 4))
        return fail(KV_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", what);
    if (q) {
        const bool in_place = q == q_out && (n_tokens == 1 || q_stride == q_out_stride);
        if ((!in_place && rows_overlap(q, q_stride * eb, qrow * eb, q_out, q_out_stride * eb, qrow * eb, n_tokens)) ||
            rows_overlap(k, k_stride * eb, krow * eb, q_out, q_out_stride * eb, qrow * eb, n_tokens) ||
            rows_overlap(v, v_stride * eb, krow * eb, q_out, q_out_stride * eb, qrow * eb, n_tokens))
            return fail(KV_ERR_INVALID_ARG, "%s: q_out overlaps q (other than in place), k or v", what);
    }
    a->seq_ids = seq_ids;
    a->slot_mapping = slot_mapping;
    a->positions = positions;
    a->q = q;
    a->q_out = q_out;
    a->k = k;
    a->v = v;
    a->k_cache = kc;
    a->v_cache = vc;
    a->q_stride = q_stride;
    a->q_out_stride = q_out_stride;
    a->k_stride = k_stride;
    a->v_stride = v_stride;
    a->positions_stride = positions_stride;
    a->n_tokens = n_tokens;
    a->num_q_heads = num_q_heads;
    a->num_kv_heads = Hkv;
    a->head_dim = D;
    a->rot_dim = rope->rot_dim;
    a->block_size = p->cfg.block_size;
    a->num_blocks = p->cfg.num_blocks;
    a->src_dtype = src_dtype;
    a->quant = quant ? 1 : 0;
    a->interleaved = rope->interleaved;
    a->pdl = 1;
    a->k_scale = k_scale;
    a->v_scale = v_scale;
    a->amplitude = rope->amplitude;
    memcpy(a->phase, rope->phase, sizeof a->phase);
    memcpy(a->axis, rope->axis, sizeof a->axis);
    uintptr_t bits = 16 | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
    if (n_tokens > 1) bits |= static_cast<uintptr_t>(k_stride * eb) | static_cast<uintptr_t>(v_stride * eb);
    if (q) {
        bits |= reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out);
        if (n_tokens > 1) bits |= static_cast<uintptr_t>(q_stride * eb) | static_cast<uintptr_t>(q_out_stride * eb);
    }
    *align = static_cast<int>(bits & (~bits + 1));
    return KV_OK;
}

kv_status_t kv_append_rope(kv_pool_t* p, int layer, const kv_rope_t* rope, const int32_t* seq_ids, int n_tokens,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride, kv_dtype_t src_dtype,
                           const int32_t* slot_mapping, const int32_t* positions, int64_t positions_stride,
                           const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int num_q_heads,
                           float k_scale, float v_scale, void* stream) {
    RopeArgs a{};
    int align = 0, sms = 0;
    if (kv_status_t st = rope_args("kv_append_rope", p, layer, rope, seq_ids, n_tokens, k, k_stride, v, v_stride,
                                   src_dtype, slot_mapping, positions, positions_stride, q, q_stride, q_out,
                                   q_out_stride, num_q_heads, k_scale, v_scale, &a, &align))
        return st;
    if (n_tokens == 0) return KV_OK;
    DeviceGuard g(p->cfg.device);
    if (!g.ok) return fail(KV_ERR_CUDA, "cannot select device %d", p->cfg.device);
    if (kv_status_t st = device_info(nullptr, &a.status, &sms, nullptr, nullptr)) return st;
    cudaError_t e = launch_append_rope(a, align, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "rope append launch");
    return KV_OK;
}

kv_status_t kv_append_norm_rope(kv_pool_t* p, int layer, const kv_rope_t* rope, const int32_t* seq_ids, int n_tokens,
                                const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                kv_dtype_t src_dtype, const int32_t* slot_mapping, const int32_t* positions,
                                int64_t positions_stride, const void* q, int64_t q_stride, void* q_out,
                                int64_t q_out_stride, int num_q_heads, const void* q_weight,
                                int64_t q_weight_stride, const void* k_weight, int64_t k_weight_stride,
                                kv_dtype_t weight_dtype, float eps, float k_scale, float v_scale, void* stream) {
    const char* what = "kv_append_norm_rope";
    NormRopeArgs a{};
    int align = 0, sms = 0;
    if (kv_status_t st = rope_args(what, p, layer, rope, seq_ids, n_tokens, k, k_stride, v, v_stride, src_dtype,
                                   slot_mapping, positions, positions_stride, q, q_stride, q_out, q_out_stride,
                                   num_q_heads, k_scale, v_scale, &a, &align))
        return st;
    const int D = p->cfg.head_dim;
    if (weight_dtype != KV_F32 && weight_dtype != src_dtype)
        return fail(KV_ERR_INVALID_ARG, "%s: weights must be KV_F32 or have the rows' dtype", what);
    if (!std::isfinite(eps) || eps < 0.f) return fail(KV_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", what);
    if (!q) q_weight = nullptr;
    const int wb = dtype_bytes(weight_dtype);
    uintptr_t wbits = 16;
    const struct {
        const void* w;
        int64_t stride;
        int heads;
    } weights[2] = {{q_weight, q_weight_stride, num_q_heads}, {k_weight, k_weight_stride, p->cfg.num_kv_heads}};
    for (const auto& x : weights) {
        if (!x.w) continue;
        if (!aligned(x.w, wb)) return fail(KV_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", what);
        if (x.heads > 1 && x.stride != 0 && x.stride < D)
            return fail(KV_ERR_INVALID_ARG, "%s: a weight stride of %lld (0, or from head_dim on)", what,
                        static_cast<long long>(x.stride));
        wbits |= reinterpret_cast<uintptr_t>(x.w) | static_cast<uintptr_t>(x.heads > 1 ? x.stride * wb : 0);
    }
    if (n_tokens == 0) return KV_OK;
    if (q) {  // a weight is read once for each token, also behind the first ones' writes to q_out
        const int64_t row = static_cast<int64_t>(num_q_heads) * D * dtype_bytes(src_dtype);
        const int64_t step = n_tokens > 1 ? q_out_stride * dtype_bytes(src_dtype) : row;
        for (const auto& x : weights) {
            const int64_t bytes = ((x.heads > 1 ? (x.heads - 1) * x.stride : 0) + D) * wb;
            if (x.w && touches_rows(x.w, bytes, q_out, step, row, n_tokens))
                return fail(KV_ERR_INVALID_ARG, "%s: q_out overlaps the weights", what);
        }
    }
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.q_weight_stride = num_q_heads > 1 ? q_weight_stride : 0;
    a.k_weight_stride = p->cfg.num_kv_heads > 1 ? k_weight_stride : 0;
    a.wide_weights = weight_dtype != src_dtype;
    a.eps = eps;
    DeviceGuard g(p->cfg.device);
    if (!g.ok) return fail(KV_ERR_CUDA, "cannot select device %d", p->cfg.device);
    if (kv_status_t st = device_info(&a.device, &a.status, &sms, nullptr, nullptr)) return st;
    cudaError_t e = launch_append_norm_rope(a, align, static_cast<int>(wbits & (~wbits + 1)), sms,
                                            static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "norm and rope append launch");
    return KV_OK;
}

static kv_status_t check_tables(const char* what, int num_seqs, int max_blocks, int block_size, int num_blocks) {
    if (num_seqs < 0 || max_blocks <= 0 || block_size <= 0 || num_blocks <= 0)
        return fail(KV_ERR_INVALID_ARG, "%s: sizes out of range", what);
    if (num_seqs > kMaxTableSeqs)
        return fail(KV_ERR_UNSUPPORTED, "%s: %d sequences (at most %d)", what, num_seqs, kMaxTableSeqs);
    if (static_cast<int64_t>(num_blocks) * block_size >= (int64_t{1} << 31) ||
        static_cast<int64_t>(max_blocks) * block_size >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "%s: slots or positions do not fit in int32", what);
    return KV_OK;
}

// Whether n words at p and m words at o can touch one another.
static bool words_overlap(const int32_t* p, int64_t n, const int32_t* o, int64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o);
    return a < b + 4 * static_cast<uintptr_t>(m) && b < a + 4 * static_cast<uintptr_t>(n);
}

kv_status_t kv_tables_extend(int32_t* block_tables, int max_blocks, const int32_t* cached_lens,
                             const int32_t* new_lens, int num_seqs, int block_size, int num_blocks,
                             const int32_t* free_queue, const int32_t* queue_state, int num_tokens,
                             int32_t* context_lens, int32_t* query_start, int32_t* slot_mapping,
                             int32_t* positions, int32_t* seq_ids, int32_t* queue_state_out, void* stream) {
    const char* what = "kv_tables_extend";
    if (kv_status_t st = check_tables(what, num_seqs, max_blocks, block_size, num_blocks)) return st;
    if (num_tokens < 0) return fail(KV_ERR_INVALID_ARG, "%s: num_tokens %d", what, num_tokens);
    if (!free_queue || !queue_state || !query_start || !queue_state_out ||
        (num_seqs > 0 && (!block_tables || !cached_lens || !new_lens || !context_lens)) ||
        (num_tokens > 0 && (!slot_mapping || !positions || !seq_ids)))
        return fail(KV_ERR_INVALID_ARG, "%s: null pointer", what);
    const int64_t B = num_seqs, T = num_tokens, M = static_cast<int64_t>(num_seqs) * max_blocks;
    // What is written, and what is read besides: no two may touch, but for an
    // input that is updated in place.
    const struct {
        const int32_t* p;
        int64_t n;
        const int32_t* may_be;  // the input that this output may stand in place of
    } out[7] = {{block_tables, M, nullptr},    {context_lens, B, cached_lens}, {query_start, B + 1, nullptr},
                {slot_mapping, T, nullptr},    {positions, T, nullptr},        {seq_ids, T, nullptr},
                {queue_state_out, 2, queue_state}};
    const struct {
        const int32_t* p;
        int64_t n;
    } in[4] = {{cached_lens, B}, {new_lens, B}, {free_queue, num_blocks}, {queue_state, 2}};
    for (int i = 0; i < 7; ++i) {
        if (!aligned(out[i].p, 4)) return fail(KV_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", what);
        if (out[i].n == 0) continue;
        for (int j = 0; j < i; ++j)
            if (out[j].n > 0 && words_overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return fail(KV_ERR_INVALID_ARG, "%s: two outputs overlap", what);
        for (const auto& x : in)
            if (x.n > 0 && !(x.p == out[i].p && x.p == out[i].may_be) && words_overlap(out[i].p, out[i].n, x.p, x.n))
                return fail(KV_ERR_INVALID_ARG, "%s: an output overlaps an input that it cannot stand in place of", what);
    }
    for (const auto& x : in)
        if (!aligned(x.p, 4)) return fail(KV_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", what);
    TablesArgs a{};
    int sms = 0;
    if (kv_status_t st = device_info(&a.device, &a.status, &sms, nullptr, nullptr)) return st;
    a.block_tables = block_tables;
    a.cached_lens = cached_lens;
    a.new_lens = new_lens;
    a.free_queue = free_queue;
    a.queue_state = queue_state;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.seq_ids = seq_ids;
    a.queue_state_out = queue_state_out;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    a.num_tokens = num_tokens;
    cudaError_t e = launch_tables_extend(a, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tables launch");
    return KV_OK;
}

kv_status_t kv_tables_release(int32_t* block_tables, int max_blocks, int32_t* context_lens, int num_seqs,
                              int block_size, int num_blocks, const int32_t* finished, int window, int sinks,
                              int32_t* free_queue, int32_t* queue_state, void* stream) {
    const char* what = "kv_tables_release";
    if (kv_status_t st = check_tables(what, num_seqs, max_blocks, block_size, num_blocks)) return st;
    if (window < 0 || sinks < 0) return fail(KV_ERR_INVALID_ARG, "%s: window %d, sinks %d", what, window, sinks);
    if (num_seqs == 0) return KV_OK;
    if (!block_tables || !context_lens || !free_queue || !queue_state)
        return fail(KV_ERR_INVALID_ARG, "%s: null pointer", what);
    const int64_t B = num_seqs, M = B * max_blocks;
    const struct {
        const int32_t* p;
        int64_t n;
    } all[5] = {{block_tables, M}, {context_lens, B}, {free_queue, num_blocks}, {queue_state, 2}, {finished, B}};
    for (int i = 0; i < 5; ++i) {
        if (!all[i].p) continue;
        if (!aligned(all[i].p, 4)) return fail(KV_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", what);
        for (int j = 0; j < i; ++j)
            if (words_overlap(all[i].p, all[i].n, all[j].p, all[j].n))
                return fail(KV_ERR_INVALID_ARG, "%s: two buffers overlap", what);
    }
    TablesArgs a{};
    if (kv_status_t st = device_info(&a.device, &a.status, nullptr, nullptr, nullptr)) return st;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.finished = finished;
    a.queue_state = queue_state;
    a.free_queue_out = free_queue;
    a.queue_state_out = queue_state;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    a.window = window;
    a.sinks = sinks;
    cudaError_t e = launch_tables_release(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tables launch");
    return KV_OK;
}

size_t kv_swap_bytes(const kv_pool_t* p, int num_blocks) {
    if (!p || num_blocks < 0) return 0;
    return static_cast<size_t>(num_blocks) * 2 * p->layer_bytes / p->cfg.num_blocks *
           p->cfg.num_layers;
}

kv_status_t kv_swap_out(const kv_pool_t* p, const int32_t* block_ids, int n, void* host_dst,
                        size_t host_bytes, void* stream) {
    return swap_blocks(const_cast<kv_pool_t*>(p), block_ids, n, host_dst, host_bytes, true, stream);
}

kv_status_t kv_swap_in(kv_pool_t* p, const int32_t* block_ids, int n, const void* host_src,
                       size_t host_bytes, void* stream) {
    return swap_blocks(p, block_ids, n, const_cast<void*>(host_src), host_bytes, false, stream);
}

kv_status_t paged_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                         int device, const kv_decode_options_t* opts, size_t* bytes) {
    if (!bytes) return fail(KV_ERR_INVALID_ARG, "null bytes_out");
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_q_heads % num_kv_heads)
        return fail(KV_ERR_INVALID_ARG, "workspace: sizes out of range");
    Options o;
    if (kv_status_t st = read_options(opts, &o)) return st;
    int sms = 0;
    if (o.num_ctas <= 0) {
        DeviceGuard g(device);
        if (!g.ok) return fail(KV_ERR_CUDA, "cannot select device %d", device);
        if (kv_status_t st = device_info(nullptr, nullptr, &sms, nullptr, nullptr)) return st;
    }
    *bytes = workspace_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, grid_size(o, sms)).total;
    return KV_OK;
}

kv_status_t paged_decode_workspace_init(void* workspace, size_t workspace_bytes, int num_seqs,
                                        int num_kv_heads, void* stream) {
    if (num_seqs < 0 || num_kv_heads <= 0) return fail(KV_ERR_INVALID_ARG, "workspace init: sizes");
    const size_t n = static_cast<size_t>(num_seqs) * num_kv_heads * 4;
    if (n == 0) return KV_OK;
    if (!workspace || workspace_bytes < n) return fail(KV_ERR_INVALID_ARG, "workspace init: buffer");
    cudaError_t e = cudaMemsetAsync(workspace, 0, n, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    return KV_OK;
}

static kv_status_t decode_impl(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                               const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                               int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                               int block_size, kv_dtype_t dtype, float scale, void* out,
                               kv_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
                               const kv_decode_options_t* opts, void* stream, const void* k_new,
                               const void* v_new, const int32_t* append_ids, int32_t* slot_out,
                               kv_dtype_t kv_dtype, float k_scale, float v_scale,
                               bool clear_counters = false, const Sight* sight = nullptr) {
    const bool fp8 = kv_dtype == KV_FP8_E4M3;
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks <= 0)
        return fail(KV_ERR_INVALID_ARG, "paged_decode_attention: sizes out of range");
    if (num_q_heads % num_kv_heads)
        return fail(KV_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                    num_kv_heads);
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8)
        return fail(KV_ERR_UNSUPPORTED, "query heads per KV head must be 1, 2, 4 or 8 (got %d)", G);
    if (head_dim != 64 && head_dim != 128) return fail(KV_ERR_UNSUPPORTED, "head_dim %d", head_dim);
    if (block_size < 1 || block_size > 256) return fail(KV_ERR_UNSUPPORTED, "block_size %d", block_size);
    if (!valid_dtype(dtype) || !valid_dtype(out_dtype))
        return fail(KV_ERR_INVALID_ARG, "unknown dtype");
    if (fp8) {
        if (dtype != KV_F16 && dtype != KV_BF16)
            return fail(KV_ERR_UNSUPPORTED, "an E4M3 cache takes an f16 or bf16 q");
        if (head_dim != 128) return fail(KV_ERR_UNSUPPORTED, "an E4M3 cache needs head_dim 128");
        if (!valid_scale(k_scale) || !valid_scale(v_scale))
            return fail(KV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
    } else if (kv_dtype != dtype) {
        return fail(KV_ERR_INVALID_ARG, "the cache must have q's dtype (or be E4M3)");
    }
    if (out_dtype != KV_F32 && out_dtype != dtype)
        return fail(KV_ERR_UNSUPPORTED, "out_dtype must be KV_F32 or the input dtype");
    if (!std::isfinite(scale)) return fail(KV_ERR_INVALID_ARG, "scale is not finite");
    if (sight) {
        if (kv_status_t st = check_sight(*sight, max_blocks, block_size)) return st;
    }
    if (static_cast<int64_t>(num_seqs) * num_kv_heads * max_blocks >= (int64_t{1} << 31) ||
        static_cast<int64_t>(num_blocks) * num_kv_heads * block_size >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "sizes exceed 32-bit tile / row indices");
    Options o;
    if (kv_status_t st = read_options(opts, &o)) return st;
    int kernel = o.kernel;
    const bool mma_ok = (dtype == KV_F16 || dtype == KV_BF16) && block_size % 16 == 0;
    if (kernel == KV_KERNEL_AUTO) kernel = mma_ok ? KV_KERNEL_MMA : KV_KERNEL_FFMA;
    if (kernel == KV_KERNEL_MMA && !mma_ok)
        return fail(KV_ERR_UNSUPPORTED, "tensor-core kernel needs f16/bf16 and block_size % 16 == 0");
    if (fp8 && kernel != KV_KERNEL_MMA)
        return fail(KV_ERR_UNSUPPORTED, "an E4M3 cache is read by the tensor-core kernel only "
                                        "(block_size a multiple of 16)");
    if (num_seqs == 0) return KV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || !workspace)
        return fail(KV_ERR_INVALID_ARG, "paged_decode_attention: null pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(workspace, 256))
        return fail(KV_ERR_INVALID_ARG,
                    "alignment: caches, q and out need 16 bytes, the workspace 256 bytes");
    if ((k_new == nullptr) != (v_new == nullptr))
        return fail(KV_ERR_INVALID_ARG, "k_new and v_new go together");
    if (k_new && (!aligned(k_new, 16) || !aligned(v_new, 16)))
        return fail(KV_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    int dev = 0, sms = 0, max_smem = 0, smem_sm = 0;
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(&dev, &status, &sms, &max_smem, &smem_sm)) return st;
    const int P = grid_size(o, sms);
    const WsLayout wl = workspace_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, P);
    if (workspace_bytes < wl.total)
        return fail(KV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes,
                    wl.total);
    // Head chunking and warps: Hc KV heads per stage, R warps per head.
    int hc = o.heads_per_stage;
    if (hc == 0) {
        hc = auto_heads_per_stage(num_kv_heads, block_size, head_dim, kv_dtype, kernel == KV_KERNEL_MMA);
    } else if (num_kv_heads % hc) {
        return fail(KV_ERR_INVALID_ARG, "heads_per_stage %d does not divide num_kv_heads %d", hc,
                    num_kv_heads);
    }
    if (kernel == KV_KERNEL_MMA && hc * block_size > 256)
        return fail(KV_ERR_UNSUPPORTED, "heads_per_stage * block_size must be <= 256 for the tensor copies");
    int R = (o.consumer_warps ? o.consumer_warps : 8) / hc;
    if (R < 1) R = 1;
    while (hc * R > 15 && R > 1) --R;
    if (hc * R > 15) return fail(KV_ERR_UNSUPPORTED, "more than 15 consumer warps");
    int budget = max_smem;
    if (o.ctas_per_sm > 1) {
        const int share = smem_sm / o.ctas_per_sm - 1024;
        if (share < budget) budget = share;
    }
    DecodePlan plan{};
    const bool planned = plan_warps(kernel, kv_dtype, head_dim, block_size, G, sight ? 2 * num_seqs : num_seqs,
                                    hc, budget, o.consumer_warps != 0, &R, &plan);
    if (!planned) return fail(KV_ERR_UNSUPPORTED, "shared memory cannot hold two stages for these sizes");

    char* ws = static_cast<char*>(workspace);
    WindowArgs a{};
    int row_blocks = max_blocks;  // the most that one query reads
    if (sight) {
        set_sight(*sight, max_blocks, block_size, &a);
        const int64_t seen = int64_t{a.sink_blocks} + a.window / block_size + 2;
        if (seen < row_blocks) row_blocks = static_cast<int>(seen);
    }
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.out = out;
    a.counters = reinterpret_cast<int32_t*>(ws + wl.counters);
    a.part_o = reinterpret_cast<float*>(ws + wl.part_o);
    a.part_ml = reinterpret_cast<float*>(ws + wl.part_ml);
    a.cum = reinterpret_cast<int32_t*>(ws + wl.cum);
    a.status = status;
    a.num_blocks = num_blocks;
    a.max_blocks = max_blocks;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.dtype = dtype;
    a.out_dtype = out_dtype;
    a.kv_dtype = kv_dtype;
    a.k_scale = fp8 ? k_scale : 1.f;
    a.v_scale = fp8 ? v_scale : 1.f;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 *
                                      static_cast<double>(a.k_scale));
    a.num_ctas = P;
    a.heads_per_stage = hc;
    a.warps_per_head = R;
    a.consumer_warps = hc * R;
    a.stages = plan.stages;
    a.smem_bytes = plan.smem_bytes;
    a.fused_reduce = o.separate_reduce ? 0 : 1;
    a.pdl = o.no_pdl ? 0 : 1;
    a.early_reads = (o.early_reads && !o.no_pdl) ? 1 : 0;
    a.test_stall = o.test_stall;
    a.phantom = phantom_items(num_seqs, num_kv_heads / hc, row_blocks, P, plan.stage_half_bytes);
    a.device = dev;
    a.k_new = k_new;
    a.v_new = v_new;
    a.append_ids = append_ids;
    a.slot_out = slot_out;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    CUtensorMap tk, tv;
    if (sight && kernel == KV_KERNEL_MMA && !(opts && (o.num_ctas || o.ctas_per_sm > 1 || o.consumer_warps || o.heads_per_stage ||
                                                       o.separate_reduce || o.test_stall))) {
        SmallPlan small{};
        const int half = block_size * head_dim * dtype_bytes(kv_dtype);
        if (plan_window_small(num_seqs, num_kv_heads, row_blocks, half, sms, max_smem, &small) &&
            small_window(small, num_seqs, num_kv_heads, row_blocks, half, fp8, sms)) {
            const int rows = num_blocks * num_kv_heads * block_size;
            if (kv_status_t st = encode_cache_map(&tk, k_cache, kv_dtype, rows, head_dim, block_size)) return st;
            if (kv_status_t st = encode_cache_map(&tv, v_cache, kv_dtype, rows, head_dim, block_size)) return st;
            a.heads_per_stage = 1;
            e = launch_window_decode_small(a, tk, tv, small, s);
            if (e != cudaSuccess) return cuda_fail(e, "windowed decode launch");
            return KV_OK;
        }
    }
    if (kernel == KV_KERNEL_MMA) {
        const int rows = num_blocks * num_kv_heads * block_size;
        if (kv_status_t st = encode_cache_map(&tk, k_cache, kv_dtype, rows, head_dim, hc * block_size)) return st;
        if (kv_status_t st = encode_cache_map(&tv, v_cache, kv_dtype, rows, head_dim, hc * block_size)) return st;
    }
    if (clear_counters) {
        e = cudaMemsetAsync(ws + wl.counters, 0, static_cast<size_t>(num_seqs) * num_kv_heads * 4, s);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    }
    if (sight) {
        e = kernel == KV_KERNEL_MMA ? launch_window_decode_mma(a, tk, tv, s) : launch_window_decode_ffma(a, s);
    } else if (kernel == KV_KERNEL_MMA) {
        e = fp8 ? launch_decode_fp8(a, tk, tv, s) : launch_decode_mma(a, tk, tv, s);
    } else {
        e = launch_decode_ffma(a, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "decode partial launch");
    if (!a.fused_reduce) {
        e = launch_decode_reduce(a, s);
        if (e != cudaSuccess) return cuda_fail(e, "decode reduce launch");
    }
    return KV_OK;
}

kv_status_t paged_decode_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                   const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                                   int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                   int block_size, kv_dtype_t dtype, float scale, void* out,
                                   kv_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
                                   const kv_decode_options_t* opts, void* stream) {
    return decode_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, context_lens, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, dtype, scale, out, out_dtype,
                       workspace, workspace_bytes, opts, stream, nullptr, nullptr, nullptr, nullptr,
                       dtype, 1.f, 1.f);
}

kv_status_t paged_decode_append_attention(const void* q, const void* k_new, const void* v_new,
                                          const int32_t* seq_ids, void* k_cache, void* v_cache,
                                          int num_blocks, const int32_t* block_tables, int max_blocks,
                                          const int32_t* context_lens, int num_seqs, int num_q_heads,
                                          int num_kv_heads, int head_dim, int block_size,
                                          kv_dtype_t dtype, float scale, void* out, kv_dtype_t out_dtype,
                                          int32_t* slot_mapping, void* workspace,
                                          size_t workspace_bytes, const kv_decode_options_t* opts,
                                          void* stream) {
    if (num_seqs > 0 && (!k_new || !v_new))
        return fail(KV_ERR_INVALID_ARG, "paged_decode_append_attention: null k_new / v_new");
    return decode_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, context_lens, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, dtype, scale, out, out_dtype,
                       workspace, workspace_bytes, opts, stream, k_new, v_new, seq_ids, slot_mapping,
                       dtype, 1.f, 1.f);
}

kv_status_t paged_decode_attention_fp8(const void* q, kv_dtype_t q_dtype, const void* k_cache,
                                       const void* v_cache, float k_scale, float v_scale, int num_blocks,
                                       const int32_t* block_tables, int max_blocks,
                                       const int32_t* context_lens, int num_seqs, int num_q_heads,
                                       int num_kv_heads, int head_dim, int block_size, float scale,
                                       void* out, kv_dtype_t out_dtype, void* workspace,
                                       size_t workspace_bytes, const kv_decode_options_t* opts,
                                       void* stream) {
    return decode_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, context_lens, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, q_dtype, scale, out, out_dtype,
                       workspace, workspace_bytes, opts, stream, nullptr, nullptr, nullptr, nullptr,
                       KV_FP8_E4M3, k_scale, v_scale);
}

kv_status_t paged_decode_append_attention_fp8(const void* q, const void* k_new, const void* v_new,
                                              const int32_t* seq_ids, kv_dtype_t q_dtype, void* k_cache,
                                              void* v_cache, float k_scale, float v_scale, int num_blocks,
                                              const int32_t* block_tables, int max_blocks,
                                              const int32_t* context_lens, int num_seqs, int num_q_heads,
                                              int num_kv_heads, int head_dim, int block_size, float scale,
                                              void* out, kv_dtype_t out_dtype, int32_t* slot_mapping,
                                              void* workspace, size_t workspace_bytes,
                                              const kv_decode_options_t* opts, void* stream) {
    if (num_seqs > 0 && (!k_new || !v_new))
        return fail(KV_ERR_INVALID_ARG, "paged_decode_append_attention_fp8: null k_new / v_new");
    return decode_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, context_lens, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, q_dtype, scale, out, out_dtype,
                       workspace, workspace_bytes, opts, stream, k_new, v_new, seq_ids, slot_mapping,
                       KV_FP8_E4M3, k_scale, v_scale);
}

kv_status_t paged_window_decode_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                          const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                                          int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                          int block_size, kv_dtype_t dtype, float scale, int window, int sinks,
                                          void* out, kv_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
                                          const kv_decode_options_t* opts, void* stream) {
    const Sight sight{window, sinks};
    return decode_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, context_lens, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, dtype, scale, out, out_dtype,
                       workspace, workspace_bytes, opts, stream, nullptr, nullptr, nullptr, nullptr,
                       dtype, 1.f, 1.f, false, &sight);
}

kv_status_t paged_window_decode_attention_fp8(const void* q, kv_dtype_t q_dtype, const void* k_cache,
                                              const void* v_cache, float k_scale, float v_scale, int num_blocks,
                                              const int32_t* block_tables, int max_blocks,
                                              const int32_t* context_lens, int num_seqs, int num_q_heads,
                                              int num_kv_heads, int head_dim, int block_size, float scale,
                                              int window, int sinks, void* out, kv_dtype_t out_dtype,
                                              void* workspace, size_t workspace_bytes,
                                              const kv_decode_options_t* opts, void* stream) {
    const Sight sight{window, sinks};
    return decode_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, context_lens, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, q_dtype, scale, out, out_dtype,
                       workspace, workspace_bytes, opts, stream, nullptr, nullptr, nullptr, nullptr,
                       KV_FP8_E4M3, k_scale, v_scale, false, &sight);
}

// ------------------------------------------------------ multi-token queries
size_t paged_prefill_workspace_bytes(int num_seqs) {
    if (num_seqs < 0) return 0;
    return align256(static_cast<size_t>(num_seqs + 1) * 4);
}

kv_status_t kv_slot_mapping_varlen(const int32_t* block_tables, int max_blocks, const int32_t* query_start,
                                   const int32_t* context_lens, int num_seqs, int num_tokens, int block_size,
                                   int num_blocks, int32_t* slot_mapping, void* stream) {
    if (num_seqs < 0 || num_tokens < 0 || max_blocks <= 0 || block_size <= 0 || num_blocks <= 0)
        return fail(KV_ERR_INVALID_ARG, "kv_slot_mapping_varlen: sizes out of range");
    if (num_seqs == 0) return KV_OK;
    if (!block_tables || !query_start || !context_lens || (num_tokens > 0 && !slot_mapping))
        return fail(KV_ERR_INVALID_ARG, "kv_slot_mapping_varlen: null pointer");
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(nullptr, &status, nullptr, nullptr, nullptr)) return st;
    PrefillArgs a{};
    a.block_tables = block_tables;
    a.query_start = query_start;
    a.context_lens = context_lens;
    a.status = status;
    a.num_blocks = num_blocks;
    a.max_blocks = max_blocks;
    a.num_seqs = num_seqs;
    a.num_tokens = num_tokens;
    a.block_size = block_size;
    a.pdl = 1;
    cudaError_t e = launch_slot_mapping_varlen(a, slot_mapping, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "varlen slot mapping launch");
    return KV_OK;
}

// The windowed prefill's: the prefix of tiles, and eight words for each tile of the tcgen05 kernel.
constexpr int kWindowRows = 256;  // rows of its tile: new tokens times query heads of a KV head
static size_t window_prefill_workspace(int num_seqs, int num_tokens, int G) {
    const size_t per = G < kWindowRows ? kWindowRows / G : 1;
    return paged_prefill_workspace_bytes(num_seqs) + align256(((num_tokens + per - 1) / per + num_seqs) * 32);
}

static kv_status_t prefill_impl(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                const int32_t* block_tables, int max_blocks, const int32_t* query_start,
                                const int32_t* context_lens, int num_seqs, int num_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int block_size, kv_dtype_t dtype,
                                kv_dtype_t kv_dtype, float k_scale, float v_scale, float scale, void* out,
                                kv_dtype_t out_dtype, void* workspace, size_t workspace_bytes, void* stream,
                                const Sight* sight = nullptr) {
    const bool fp8 = kv_dtype == KV_FP8_E4M3;
    if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
        max_blocks <= 0)
        return fail(KV_ERR_INVALID_ARG, "paged_prefill_attention: sizes out of range");
    if (num_q_heads % num_kv_heads)
        return fail(KV_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                    num_kv_heads);
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8)
        return fail(KV_ERR_UNSUPPORTED, "query heads per KV head must be 1, 2, 4 or 8 (got %d)", G);
    if (head_dim != 64 && head_dim != 128) return fail(KV_ERR_UNSUPPORTED, "head_dim %d", head_dim);
    if (dtype == KV_F32 && !fp8) {
        if (block_size < 1 || block_size > 256)
            return fail(KV_ERR_UNSUPPORTED, "block_size must be 1 .. 256");
    } else if (block_size % 16 || block_size < 16 || block_size > 256) {
        return fail(KV_ERR_UNSUPPORTED, "multi-token queries on f16/bf16 need block_size a multiple of 16 up to 256");
    }
    if (fp8) {
        if (dtype != KV_F16 && dtype != KV_BF16)
            return fail(KV_ERR_UNSUPPORTED, "an E4M3 cache takes an f16 or bf16 q");
        if (head_dim != 128) return fail(KV_ERR_UNSUPPORTED, "an E4M3 cache needs head_dim 128");
        if (!valid_scale(k_scale) || !valid_scale(v_scale))
            return fail(KV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
    } else if (dtype != KV_F32 && dtype != KV_F16 && dtype != KV_BF16) {
        return fail(KV_ERR_INVALID_ARG, "unknown dtype");
    }
    if (out_dtype != KV_F32 && out_dtype != dtype)
        return fail(KV_ERR_UNSUPPORTED, "out_dtype must be KV_F32 or the input dtype");
    if (!std::isfinite(scale)) return fail(KV_ERR_INVALID_ARG, "scale is not finite");
    if (sight) {
        if (kv_status_t st = check_sight(*sight, max_blocks, block_size)) return st;
    }
    if (static_cast<int64_t>(num_blocks) * num_kv_heads * block_size >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "sizes exceed 32-bit row indices");
    if (num_seqs == 0 || num_tokens == 0) return KV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens || !out || !workspace)
        return fail(KV_ERR_INVALID_ARG, "paged_prefill_attention: null pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16))
        return fail(KV_ERR_INVALID_ARG, "alignment: caches, q, out and the workspace need 16 bytes");
    const size_t need = sight ? window_prefill_workspace(num_seqs, num_tokens, G) : paged_prefill_workspace_bytes(num_seqs);
    if (workspace_bytes < need)
        return fail(KV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (sight) {  // (rows computed again read q after out has been written)
        const uintptr_t n = static_cast<uintptr_t>(num_tokens) * num_q_heads * head_dim;
        const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
        if (q0 < o0 + n * dtype_bytes(out_dtype) && o0 < q0 + n * dtype_bytes(dtype))
            return fail(KV_ERR_INVALID_ARG, "paged_window_prefill_attention: out overlaps q");
    }
    int dev = 0, sms = 0, max_smem = 0;
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(&dev, &status, &sms, &max_smem, nullptr)) return st;
    // The tcgen05 kernel: f16/bf16 cache, head_dim 128, blocks that tile 64-key tiles evenly.
    const bool tc = !sight && !fp8 && dtype != KV_F32 && head_dim == 128 &&
                    (block_size % 64 == 0 || 64 % block_size == 0) && prefill_tc_smem_bytes() <= max_smem;
    // Stages of the warp-MMA kernel hold K and V in q's 2-byte type (an E4M3
    // block converted); E4M3 adds two raw slots of codes.
    const int stage_bytes = 2 * block_size * head_dim * 2;
    const int raw_bytes = fp8 ? 4 * block_size * head_dim : 0;
    int stages = (max_smem - 2048 - 64 - raw_bytes) / stage_bytes;
    if (stages > 4) stages = 4;
    const bool window_tc = sight && dtype != KV_F32;
    if (!tc && !window_tc && dtype != KV_F32 && stages < 2) return fail(KV_ERR_UNSUPPORTED, "shared memory cannot hold two stages");
    PrefillArgs a{};
    if (sight) set_sight(*sight, max_blocks, block_size, &a);
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.query_start = query_start;
    a.context_lens = context_lens;
    a.out = out;
    a.tile_cum = static_cast<int32_t*>(workspace);
    a.status = status;
    a.num_blocks = num_blocks;
    a.max_blocks = max_blocks;
    a.num_seqs = num_seqs;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.dtype = dtype;
    a.out_dtype = out_dtype;
    a.kv_dtype = fp8 ? KV_FP8_E4M3 : dtype;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 *
                                      static_cast<double>(fp8 ? k_scale : 1.f));
    a.v_scale = fp8 ? v_scale : 1.f;
    a.stages = stages;
    a.smem_bytes = tc ? prefill_tc_smem_bytes()
                      : fp8 ? 1024 + stages * stage_bytes + 1024 + raw_bytes
                            : 1024 + stages * stage_bytes + stages * 16 + 32;
    a.tensor_cores = tc ? 1 : 0;
    a.tile_tokens = window_tc ? kWindowRows / G : tc ? 128 / G : 16;
    const int64_t tiles = (static_cast<int64_t>(num_tokens) + a.tile_tokens - 1) / a.tile_tokens + num_seqs;
    if (tiles >= (int64_t{1} << 31)) return fail(KV_ERR_UNSUPPORTED, "too many query tiles");
    a.grid_tiles = static_cast<int>(tiles);
    a.pdl = 1;
    a.device = dev;
    CUtensorMap tk{}, tv{};
    if (window_tc) {
        a.smem_bytes = window_prefill_tc_smem_bytes(head_dim);
        if (a.smem_bytes > max_smem) return fail(KV_ERR_UNSUPPORTED, "%d bytes of shared memory needed", a.smem_bytes);
        a.tiles = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + paged_prefill_workspace_bytes(num_seqs));
        a.box = block_size % 32 ? 16 : 32;
        const int rows = num_blocks * num_kv_heads * block_size;
        CUtensorMap tq{};
        if (kv_status_t st = encode_query_map(&tq, q, dtype, num_tokens, num_q_heads, head_dim, G, 128 / G)) return st;
        if (!fp8) {  // (E4M3 codes come by bulk copies)
            if (kv_status_t st = encode_group_map(&tk, k_cache, dtype, rows, head_dim, a.box)) return st;
            if (kv_status_t st = encode_group_map(&tv, v_cache, dtype, rows, head_dim, a.box)) return st;
        }
        cudaError_t e = launch_window_prefill_tc(a, tq, tk, tv, sms, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return cuda_fail(e, "windowed prefill launch");
        return KV_OK;
    }
    if (!fp8 && dtype != KV_F32) {  // E4M3 tiles come by bulk copies, f32 rows by plain loads
        const int rows = num_blocks * num_kv_heads * block_size;
        const int box_rows = tc ? (block_size < 64 ? block_size : 64) : block_size;
        if (kv_status_t st = encode_cache_map(&tk, k_cache, dtype, rows, head_dim, box_rows)) return st;
        if (kv_status_t st = encode_cache_map(&tv, v_cache, dtype, rows, head_dim, box_rows)) return st;
    }
    cudaError_t e = launch_prefill(a, tk, tv, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
    return KV_OK;
}

kv_status_t paged_prefill_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                    const int32_t* block_tables, int max_blocks, const int32_t* query_start,
                                    const int32_t* context_lens, int num_seqs, int num_tokens, int num_q_heads,
                                    int num_kv_heads, int head_dim, int block_size, kv_dtype_t dtype,
                                    float scale, void* out, kv_dtype_t out_dtype, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    if (dtype == KV_FP8_E4M3)
        return fail(KV_ERR_INVALID_ARG, "paged_prefill_attention: an E4M3 cache goes to paged_prefill_attention_fp8");
    return prefill_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, query_start, context_lens,
                        num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, dtype, dtype, 1.f,
                        1.f, scale, out, out_dtype, workspace, workspace_bytes, stream);
}

kv_status_t paged_prefill_attention_fp8(const void* q, kv_dtype_t q_dtype, const void* k_cache,
                                        const void* v_cache, float k_scale, float v_scale, int num_blocks,
                                        const int32_t* block_tables, int max_blocks, const int32_t* query_start,
                                        const int32_t* context_lens, int num_seqs, int num_tokens,
                                        int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                        float scale, void* out, kv_dtype_t out_dtype, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    return prefill_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, query_start, context_lens,
                        num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, q_dtype,
                        KV_FP8_E4M3, k_scale, v_scale, scale, out, out_dtype, workspace, workspace_bytes, stream);
}

kv_status_t paged_window_prefill_workspace_bytes(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                                                 int head_dim, int device, size_t* bytes) {
    if (!bytes) return fail(KV_ERR_INVALID_ARG, "null bytes_out");
    if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || device < 0 ||
        num_q_heads % num_kv_heads)
        return fail(KV_ERR_INVALID_ARG, "workspace: sizes out of range");
    *bytes = window_prefill_workspace(num_seqs, num_tokens, num_q_heads / num_kv_heads);
    return KV_OK;
}

kv_status_t paged_window_prefill_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                           const int32_t* block_tables, int max_blocks, const int32_t* query_start,
                                           const int32_t* context_lens, int num_seqs, int num_tokens,
                                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                           kv_dtype_t dtype, float scale, int window, int sinks, void* out,
                                           kv_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
                                           void* stream) {
    if (dtype == KV_FP8_E4M3)
        return fail(KV_ERR_INVALID_ARG,
                    "paged_window_prefill_attention: an E4M3 cache goes to paged_window_prefill_attention_fp8");
    const Sight sight{window, sinks};
    return prefill_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, query_start, context_lens,
                        num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, dtype, dtype, 1.f,
                        1.f, scale, out, out_dtype, workspace, workspace_bytes, stream, &sight);
}

kv_status_t paged_window_prefill_attention_fp8(const void* q, kv_dtype_t q_dtype, const void* k_cache,
                                               const void* v_cache, float k_scale, float v_scale, int num_blocks,
                                               const int32_t* block_tables, int max_blocks,
                                               const int32_t* query_start, const int32_t* context_lens,
                                               int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                                               int head_dim, int block_size, float scale, int window, int sinks,
                                               void* out, kv_dtype_t out_dtype, void* workspace,
                                               size_t workspace_bytes, void* stream) {
    const Sight sight{window, sinks};
    return prefill_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, query_start, context_lens,
                        num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, q_dtype,
                        KV_FP8_E4M3, k_scale, v_scale, scale, out, out_dtype, workspace, workspace_bytes, stream,
                        &sight);
}

// ------------------------------------------------------- shared prefixes
namespace {

struct SharedWs {
    size_t parts, tails, part_o, part_ml, total;
    int max_rows;
};

SharedWs shared_workspace(int B, int Hq, int Hkv, int D, int sms) {
    SharedWs w;
    // 128 rows for each CTA's share of the work, and two parts more of every
    // row (see prefix_units.cuh); then the tails' partials (WsLayout).
    w.max_rows = static_cast<int>(int64_t{128} * sms + 2 * static_cast<int64_t>(B) * Hq);
    const size_t rows = static_cast<size_t>(w.max_rows) + (static_cast<size_t>(sms) + B) * Hq;
    w.parts = 0;
    w.tails = align256(static_cast<size_t>(B) * Hkv * sizeof(int4));
    w.part_o = w.tails + align256(static_cast<size_t>(B) * Hkv * sizeof(int4));
    w.part_ml = w.part_o + align256(rows * D * 4);
    w.total = w.part_ml + align256(rows * 8);
    return w;
}

kv_status_t shared_sizes(const char* what, int B, int ng, int Hq, int Hkv, int D) {
    if (B < 0 || ng < 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return fail(KV_ERR_INVALID_ARG, "%s: sizes out of range", what);
    if (Hq % Hkv) return fail(KV_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d", Hq, Hkv);
    if (static_cast<int64_t>(B) * Hq >= (int64_t{1} << 29) || static_cast<int64_t>(ng) * Hkv >= (int64_t{1} << 24))
        return fail(KV_ERR_UNSUPPORTED, "%s: too many sequences or groups", what);
    return KV_OK;
}

kv_status_t shared_prefix_impl(const void* q, kv_dtype_t dtype, const void* k_cache, const void* v_cache,
                               kv_dtype_t kv_dtype, float k_scale, float v_scale, int num_blocks,
                               const int32_t* block_tables, int max_blocks, const int32_t* context_lens, int num_seqs,
                               const int32_t* group_start, const int32_t* prefix_lens, int num_groups,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale, void* out,
                               kv_dtype_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const char* what = "paged_shared_prefix_attention";
    const bool fp8 = kv_dtype == KV_FP8_E4M3;
    if (kv_status_t st = shared_sizes(what, num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim)) return st;
    if (num_blocks <= 0 || max_blocks <= 0) return fail(KV_ERR_INVALID_ARG, "%s: sizes out of range", what);
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8)
        return fail(KV_ERR_UNSUPPORTED, "query heads per KV head must be 1, 2, 4 or 8 (got %d)", G);
    if (head_dim != 64 && head_dim != 128) return fail(KV_ERR_UNSUPPORTED, "head_dim %d", head_dim);
    if (block_size < 16 || block_size > 256 || block_size % 16)
        return fail(KV_ERR_UNSUPPORTED, "%s needs block_size a multiple of 16 up to 256 (got %d)", what, block_size);
    if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return fail(KV_ERR_INVALID_ARG, "unknown dtype");
    if (dtype == KV_F32) return fail(KV_ERR_UNSUPPORTED, "%s takes f16 or bf16", what);
    if (fp8) {
        if (head_dim != 128) return fail(KV_ERR_UNSUPPORTED, "an E4M3 cache needs head_dim 128");
        if (!valid_scale(k_scale) || !valid_scale(v_scale))
            return fail(KV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
    }
    if (out_dtype != KV_F32 && out_dtype != dtype)
        return fail(KV_ERR_UNSUPPORTED, "out_dtype must be KV_F32 or the input dtype");
    if (!std::isfinite(scale)) return fail(KV_ERR_INVALID_ARG, "scale is not finite");
    if (static_cast<int64_t>(num_seqs) * num_kv_heads * max_blocks >= (int64_t{1} << 31) ||
        static_cast<int64_t>(max_blocks) * block_size >= (int64_t{1} << 31) - 64 ||
        static_cast<int64_t>(num_blocks) * num_kv_heads * block_size >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "sizes exceed 32-bit tile / row indices");
    // Key tiles of all rows of the prefix part, at most.
    if (((static_cast<int64_t>(num_seqs) * G / 128 + num_groups) * num_kv_heads) *
            (static_cast<int64_t>(max_blocks) * block_size / 64 + 1) >= (int64_t{1} << 31))
        return fail(KV_ERR_UNSUPPORTED, "%s: more than 2^31 tiles of work", what);
    if (num_seqs == 0) return KV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || !workspace ||
        (num_groups > 0 && (!group_start || !prefix_lens)))
        return fail(KV_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(workspace, 256))
        return fail(KV_ERR_INVALID_ARG,
                    "alignment: caches, q and out need 16 bytes, the workspace 256 bytes");
    if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(group_start, 4) || !aligned(prefix_lens, 4))
        return fail(KV_ERR_INVALID_ARG, "%s: an int32 array is not 4-byte aligned", what);
    int dev = 0, sms = 0, max_smem = 0;
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(&dev, &status, &sms, &max_smem, nullptr)) return st;
    max_smem -= prefix_static_smem_bytes();
    const SharedWs w = shared_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, sms);
    if (workspace_bytes < w.total)
        return fail(KV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, w.total);
    // The tails: heads a stage as the decode kernel's default, up to 11 (its
    // variant for partials is built for 12 warps).
    int hc = auto_heads_per_stage(num_kv_heads, block_size, head_dim, kv_dtype, true);
    while (hc > 11 || num_kv_heads % hc) --hc;
    int R = 8 / hc > 1 ? 8 / hc : 1;
    DecodePlan plan{};
    // (Room in shared memory for each sequence's shared blocks besides its place.)
    if (!plan_warps(KV_KERNEL_MMA, kv_dtype, head_dim, block_size, G, 2 * num_seqs, hc, max_smem, false, &R, &plan))
        return fail(KV_ERR_UNSUPPORTED, "shared memory cannot hold two stages for these sizes");

    char* ws = static_cast<char*>(workspace);
    SharedPrefixArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.group_start = group_start;
    a.prefix_lens = prefix_lens;
    a.out = out;
    a.status = status;
    a.parts = reinterpret_cast<int4*>(ws + w.parts);
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
    a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
    a.num_seqs = num_seqs;
    a.num_groups = num_groups;
    a.num_blocks = num_blocks;
    a.max_blocks = max_blocks;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.dtype = dtype;
    a.out_dtype = out_dtype;
    a.kv_dtype = kv_dtype;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 *
                                      static_cast<double>(fp8 ? k_scale : 1.f));
    a.v_scale = fp8 ? v_scale : 1.f;
    a.max_rows = w.max_rows;
    const int parts_smem = prefix_smem_bytes(head_dim, fp8);
    if (parts_smem > max_smem) return fail(KV_ERR_UNSUPPORTED, "%s: not enough shared memory on this device", what);

    TailArgs d{};
    d.q = q;
    d.k_cache = k_cache;
    d.v_cache = v_cache;
    d.block_tables = block_tables;
    d.context_lens = context_lens;
    d.group_start = group_start;
    d.prefix_lens = prefix_lens;
    d.num_groups = num_groups;
    d.tail_parts = reinterpret_cast<int4*>(ws + w.tails);
    d.prefix_parts = a.parts;
    d.out = out;
    d.part_o = a.part_o + static_cast<size_t>(w.max_rows) * head_dim;
    d.part_ml = a.part_ml + static_cast<size_t>(w.max_rows) * 2;
    d.status = status;
    d.num_blocks = num_blocks;
    d.max_blocks = max_blocks;
    d.num_seqs = num_seqs;
    d.num_q_heads = num_q_heads;
    d.num_kv_heads = num_kv_heads;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.dtype = dtype;
    d.out_dtype = out_dtype;
    d.kv_dtype = kv_dtype;
    d.k_scale = fp8 ? k_scale : 1.f;
    d.v_scale = a.v_scale;
    d.scale_log2 = a.scale_log2;
    d.num_ctas = sms;
    d.heads_per_stage = hc;
    d.warps_per_head = R;
    d.consumer_warps = hc * R;
    d.stages = plan.stages;
    d.smem_bytes = plan.smem_bytes > parts_smem ? plan.smem_bytes : parts_smem;
    d.fused_reduce = 0;
    d.pdl = 1;
    d.phantom = phantom_items(num_seqs, num_kv_heads / hc, max_blocks, sms, plan.stage_half_bytes);
    d.device = dev;
    CUtensorMap tk, tv;
    const int rows = num_blocks * num_kv_heads * block_size;
    if (kv_status_t st = encode_cache_map(&tk, k_cache, kv_dtype, rows, head_dim, hc * block_size)) return st;
    if (kv_status_t st = encode_cache_map(&tv, v_cache, kv_dtype, rows, head_dim, hc * block_size)) return st;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_shared_prefix(a, d, tk, tv, s);
    if (e != cudaSuccess) return cuda_fail(e, "shared-prefix launch");
    return KV_OK;
}

}  // namespace

kv_status_t paged_shared_prefix_workspace_bytes(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads,
                                                int head_dim, int device, size_t* bytes) {
    if (!bytes) return fail(KV_ERR_INVALID_ARG, "null bytes_out");
    if (kv_status_t st = shared_sizes("shared-prefix workspace", num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim))
        return st;
    DeviceGuard g(device);
    if (!g.ok) return fail(KV_ERR_CUDA, "cannot select device %d", device);
    int sms = 0;
    if (kv_status_t st = device_info(nullptr, nullptr, &sms, nullptr, nullptr)) return st;
    *bytes = shared_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, sms).total;
    return KV_OK;
}

kv_status_t paged_shared_prefix_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                          const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                                          int num_seqs, const int32_t* group_start, const int32_t* prefix_lens,
                                          int num_groups, int num_q_heads, int num_kv_heads, int head_dim,
                                          int block_size, kv_dtype_t dtype, float scale, void* out,
                                          kv_dtype_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype == KV_FP8_E4M3)
        return fail(KV_ERR_INVALID_ARG, "paged_shared_prefix_attention: an E4M3 cache goes to paged_shared_prefix_attention_fp8");
    return shared_prefix_impl(q, dtype, k_cache, v_cache, dtype, 1.f, 1.f, num_blocks, block_tables, max_blocks,
                              context_lens, num_seqs, group_start, prefix_lens, num_groups, num_q_heads, num_kv_heads,
                              head_dim, block_size, scale, out, out_dtype, workspace, workspace_bytes, stream);
}

kv_status_t paged_shared_prefix_attention_fp8(const void* q, kv_dtype_t q_dtype, const void* k_cache,
                                              const void* v_cache, float k_scale, float v_scale, int num_blocks,
                                              const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                                              int num_seqs, const int32_t* group_start, const int32_t* prefix_lens,
                                              int num_groups, int num_q_heads, int num_kv_heads, int head_dim,
                                              int block_size, float scale, void* out, kv_dtype_t out_dtype,
                                              void* workspace, size_t workspace_bytes, void* stream) {
    return shared_prefix_impl(q, q_dtype, k_cache, v_cache, KV_FP8_E4M3, k_scale, v_scale, num_blocks, block_tables,
                              max_blocks, context_lens, num_seqs, group_start, prefix_lens, num_groups, num_q_heads,
                              num_kv_heads, head_dim, block_size, scale, out, out_dtype, workspace, workspace_bytes,
                              stream);
}

kv_status_t kv_device_status(int device, void* stream, uint32_t* flags_out) {
    DeviceGuard g(device);
    if (!g.ok) return fail(KV_ERR_CUDA, "cannot select device %d", device);
    uint32_t* status = nullptr;
    if (kv_status_t st = device_info(nullptr, &status, nullptr, nullptr, nullptr)) return st;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    uint32_t flags = 0;
    if ((e = cudaMemcpy(&flags, status, sizeof flags, cudaMemcpyDeviceToHost)) != cudaSuccess)
        return cuda_fail(e, "reading the status word");
    if (flags && (e = cudaMemset(status, 0, sizeof flags)) != cudaSuccess)
        return cuda_fail(e, "clearing the status word");
    if (flags_out) *flags_out = flags;
    if (!flags) return KV_OK;
    if (flags & KV_FLAG_TIMEOUT) return fail(KV_ERR_DEVICE_TIMEOUT, "a kernel gave up a bounded wait");
    return fail(KV_ERR_DEVICE_CHECK, "device check flags 0x%x", flags);
}

// ------------------------------------------------------------ allocator
kv_status_t kv_allocator_create(int num_blocks, int block_size, int reserve_null_block,
                                kv_block_allocator_t** out) {
    if (!out) return fail(KV_ERR_INVALID_ARG, "null out");
    *out = nullptr;
    if (num_blocks <= 0 || block_size <= 0) return fail(KV_ERR_INVALID_ARG, "allocator sizes");
    kv_block_allocator* a = new (std::nothrow) kv_block_allocator;
    if (!a) return fail(KV_ERR_OUT_OF_MEMORY, "host allocation failed");
    a->num_blocks = num_blocks;
    a->block_size = block_size;
    for (int b = reserve_null_block ? 1 : 0; b < num_blocks; ++b) a->free_q.push_back(b);
    *out = a;
    return KV_OK;
}

void kv_allocator_destroy(kv_block_allocator_t* a) { delete a; }

kv_status_t kv_allocator_extend(kv_block_allocator_t* a, int64_t seq_id, int new_tokens) {
    if (!a || new_tokens < 0) return fail(KV_ERR_INVALID_ARG, "kv_allocator_extend arguments");
    auto it = a->seqs.find(seq_id);
    const int64_t have_tokens = it == a->seqs.end() ? 0 : it->second.tokens;
    const size_t have_blocks = it == a->seqs.end() ? 0 : it->second.table.size();
    const int64_t total = have_tokens + new_tokens;
    const int64_t need_blocks = (total + a->block_size - 1) / a->block_size - static_cast<int64_t>(have_blocks);
    if (need_blocks > static_cast<int64_t>(a->free_q.size()))
        return fail(KV_ERR_OUT_OF_BLOCKS, "sequence %lld needs %lld blocks, %zu free",
                    static_cast<long long>(seq_id), static_cast<long long>(need_blocks), a->free_q.size());
    auto& s = a->seqs[seq_id];
    for (int64_t i = 0; i < need_blocks; ++i) {
        s.table.push_back(a->free_q.front());
        a->free_q.pop_front();
    }
    s.tokens = total;
    return KV_OK;
}

kv_status_t kv_allocator_release(kv_block_allocator_t* a, int64_t seq_id) {
    if (!a) return fail(KV_ERR_INVALID_ARG, "null allocator");
    auto it = a->seqs.find(seq_id);
    if (it == a->seqs.end()) return fail(KV_ERR_NOT_FOUND, "unknown sequence %lld", static_cast<long long>(seq_id));
    for (int32_t b : it->second.table) a->free_q.push_back(b);
    a->seqs.erase(it);
    return KV_OK;
}

kv_status_t kv_allocator_table(const kv_block_allocator_t* a, int64_t seq_id, int32_t* table_out,
                               int capacity, int* num_blocks_out, int* num_tokens_out) {
    if (!a || capacity < 0 || (capacity > 0 && !table_out)) return fail(KV_ERR_INVALID_ARG, "kv_allocator_table arguments");
    auto it = a->seqs.find(seq_id);
    if (it == a->seqs.end()) return fail(KV_ERR_NOT_FOUND, "unknown sequence %lld", static_cast<long long>(seq_id));
    const auto& t = it->second.table;
    if (static_cast<int>(t.size()) > capacity && table_out)
        return fail(KV_ERR_INVALID_ARG, "table of %zu blocks does not fit in %d entries", t.size(), capacity);
    for (size_t i = 0; i < t.size() && table_out; ++i) table_out[i] = t[i];
    if (num_blocks_out) *num_blocks_out = static_cast<int>(t.size());
    if (num_tokens_out) *num_tokens_out = static_cast<int>(it->second.tokens);
    return KV_OK;
}

kv_status_t kv_allocator_slot(const kv_block_allocator_t* a, int64_t seq_id, int position, int32_t* slot_out) {
    if (!a || !slot_out) return fail(KV_ERR_INVALID_ARG, "kv_allocator_slot arguments");
    auto it = a->seqs.find(seq_id);
    if (it == a->seqs.end()) return fail(KV_ERR_NOT_FOUND, "unknown sequence %lld", static_cast<long long>(seq_id));
    const auto& t = it->second.table;
    if (position < 0 || static_cast<int64_t>(position) >= static_cast<int64_t>(t.size()) * a->block_size)
        return fail(KV_ERR_INVALID_ARG, "position %d outside the sequence's blocks", position);
    *slot_out = t[position / a->block_size] * a->block_size + position % a->block_size;
    return KV_OK;
}

kv_status_t kv_seq_extend(kv_pool_t* p, int seq_id, int new_tokens, int32_t* table_row, int max_blocks,
                          int* ctx_len_inout, int32_t* slot_out) {
    if (!p || !table_row || !ctx_len_inout || max_blocks <= 0 || new_tokens < 0 || (new_tokens > 0 && !slot_out))
        return fail(KV_ERR_INVALID_ARG, "kv_seq_extend arguments");
    if (!p->alloc) {
        if (kv_status_t st = kv_allocator_create(p->cfg.num_blocks, p->cfg.block_size, 0, &p->alloc)) return st;
    }
    kv_block_allocator* a = p->alloc;
    auto it = a->seqs.find(seq_id);
    const int64_t have = it == a->seqs.end() ? 0 : it->second.tokens;
    if (*ctx_len_inout != have)
        return fail(KV_ERR_INVALID_ARG, "sequence %d holds %lld tokens, the caller says %d", seq_id,
                    static_cast<long long>(have), *ctx_len_inout);
    const int64_t total = have + new_tokens;
    const int64_t blocks = (total + a->block_size - 1) / a->block_size;
    if (blocks > max_blocks)
        return fail(KV_ERR_INVALID_ARG, "sequence %d would need %lld table entries, %d given", seq_id,
                    static_cast<long long>(blocks), max_blocks);
    if (kv_status_t st = kv_allocator_extend(a, seq_id, new_tokens)) return st;
    const auto& t = a->seqs[seq_id].table;
    for (int i = 0; i < max_blocks; ++i) table_row[i] = i < static_cast<int>(t.size()) ? t[i] : -1;
    for (int i = 0; i < new_tokens; ++i) {
        const int64_t pos = have + i;
        slot_out[i] = t[pos / a->block_size] * a->block_size + static_cast<int32_t>(pos % a->block_size);
    }
    *ctx_len_inout = static_cast<int>(total);
    return KV_OK;
}

kv_status_t kv_seq_free(kv_pool_t* p, int seq_id) {
    if (!p) return fail(KV_ERR_INVALID_ARG, "null pool");
    if (!p->alloc) return fail(KV_ERR_NOT_FOUND, "unknown sequence %d", seq_id);
    return kv_allocator_release(p->alloc, seq_id);
}

kv_status_t kv_allocator_free_queue(const kv_block_allocator_t* a, int32_t* out, int capacity, int* count_out) {
    if (!a || capacity < 0 || (capacity > 0 && !out)) return fail(KV_ERR_INVALID_ARG, "kv_allocator_free_queue arguments");
    const int n = static_cast<int>(a->free_q.size());
    if (count_out) *count_out = n;
    if (out) {
        if (n > capacity) return fail(KV_ERR_INVALID_ARG, "free queue of %d does not fit in %d", n, capacity);
        int i = 0;
        for (int32_t b : a->free_q) out[i++] = b;
    }
    return KV_OK;
}

}  // extern "C"

namespace pkv {
kv_status_t decode_attention_clearing_counters(const void* q, const void* k_cache, const void* v_cache,
                                               int num_blocks, const int32_t* block_tables, int max_blocks,
                                               const int32_t* context_lens, int num_seqs, int num_q_heads,
                                               int num_kv_heads, int head_dim, int block_size, int dtype,
                                               float scale, void* out, int out_dtype, void* workspace,
                                               size_t workspace_bytes, const void* opts, void* stream) {
    const kv_dtype_t dt = static_cast<kv_dtype_t>(dtype);
    return decode_impl(q, k_cache, v_cache, num_blocks, block_tables, max_blocks, context_lens, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, dt, scale, out,
                       static_cast<kv_dtype_t>(out_dtype), workspace, workspace_bytes,
                       static_cast<const kv_decode_options_t*>(opts), stream, nullptr, nullptr, nullptr,
                       nullptr, dt, 1.f, 1.f, /*clear_counters=*/true);
}
}  // namespace pkv
