// pa_sparse.h -- types and launchers of the sparse decode step: tables of a step, bounds of keys, selection of
// blocks, attention over the selected blocks.
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int STATUS_NO_BLOCKS = 4;   // device status word: a step needed more blocks than were free

struct TablesParams {
    int num_seqs, num_tokens;
    int32_t *block_tables;
    int64_t stride;
    int32_t *context_lens;
    const int32_t *keep_lens;   // NULL: nothing is cut back
    const int32_t *new_lens;
    int32_t *free_blocks, *num_free;
    int32_t *cu_q, *positions;
    int64_t *slots;
    int bs_shift;
    int num_blocks;
    int max_len;                // longest context the tables hold
    bool vectors;               // positions and slots lie on 16-byte boundaries
    bool tokens_apart;          // positions and slots are written by a kernel behind the one that makes the tables
    int *status;
};

struct BoundsParams {
    const void *k_cache;
    const float *k_scales;      // FP8 pools: per (slot, head)
    const int32_t *cu_q;
    const int32_t *block_tables;
    int64_t stride;
    const int32_t *context_lens;
    int num_tokens, num_seqs;
    int Hkv, bs, num_blocks, max_len;
    int8_t *codes;              // [num_blocks, Hkv, 2, head_dim]
    float *steps;               // [num_blocks, Hkv]
    int *status;
};

struct SelectParams {
    const void *q;
    const int8_t *codes;
    const float *steps;
    const int32_t *block_tables;
    int64_t stride;
    const int32_t *context_lens;
    int num_seqs, Hq, Hkv, G, q_len, rows;
    int bs, num_blocks, max_len;
    int budget, num_first, num_last;
    int chunk;                  // blocks that one CTA of a cluster scores, a multiple of 16
    int32_t *selected;
    int *status;
};

struct SelectedParams {
    const void *q;
    void *out;
    const float *k_scales, *v_scales;   // FP8 pools
    const int32_t *selected;
    int budget;
    const int32_t *block_tables;
    int64_t stride;
    const int32_t *context_lens;
    int num_seqs, Hq, Hkv, G, q_len, rows;
    int bs, num_blocks, max_len;
    int warp_tiles;             // entries of a warp's tile list
    float scale_log2;
    uint64_t wait_ns;
    int *status;
};

cudaError_t launch_tables(TablesParams p, int sm_count, cudaStream_t stream);
cudaError_t launch_key_bounds(const BoundsParams &p, int dtype, int head_dim, int sm_count, cudaStream_t stream);
cudaError_t launch_select(SelectParams p, int dtype, int head_dim, int sm_count, cudaStream_t stream);
cudaError_t launch_selected(SelectedParams p, int dtype, int head_dim, const CUtensorMap &tmk, const CUtensorMap &tmv,
                            int sm_count, cudaStream_t stream);

// A launch as clusters of `cluster` CTAs, behind the kernel ahead of it in the stream (as launch_pdl).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, int cluster,
                                   cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

}  // namespace pa
