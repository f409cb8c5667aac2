// Shared between the kernels of the shared-prefix attention and its host side.
#pragma once

#include "pkv_internal.h"

namespace pkv {

struct SharedPrefixArgs {
    const void* q;               // [B][Hq][D]
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* group_start;  // [num_groups + 1]
    const int32_t* prefix_lens;  // [num_groups]
    void* out;
    uint32_t* status;
    // Workspace.
    int4* parts;                 // [B][Hkv] (x, y, z, -): part k < z of query head g of the KV head is
                                 // partial row x + k * y + g
    float* part_o;               // [max_rows, then the tails'][D]
    float* part_ml;              // [max_rows, then the tails'][2]
    int num_seqs, num_groups, num_blocks, max_blocks, num_q_heads, num_kv_heads, head_dim, block_size;
    int dtype, out_dtype, kv_dtype;
    float scale_log2, v_scale;
    int max_rows;                // capacity of the partial rows
};

// Shared memory of the parts role: dynamic, and what the kernel holds besides.
int prefix_static_smem_bytes();
int prefix_smem_bytes(int head_dim, bool fp8);
cudaError_t launch_attend_f16(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmap_k,
                              const CUtensorMap& tmap_v, cudaStream_t stream);
cudaError_t launch_attend_bf16(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmap_k,
                               const CUtensorMap& tmap_v, cudaStream_t stream);
cudaError_t launch_attend_fp8(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmap_k,
                              const CUtensorMap& tmap_v, cudaStream_t stream);
cudaError_t launch_shared_prefix(const SharedPrefixArgs& a, const TailArgs& d, const CUtensorMap& tmap_k,
                                 const CUtensorMap& tmap_v, cudaStream_t stream);

}  // namespace pkv
