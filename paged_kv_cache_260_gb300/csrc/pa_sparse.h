// pa_sparse.h -- what the host side of the block-selection, weight-accounting
// and eviction entry points shares with their kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pa {

// pa_block_bounds: the least and greatest key of every channel of a block.
struct BoundsParams {
    const void *k_cache;
    void *bounds;                  // [num_blocks][num_kv_heads][2][head_dim]
    const int32_t *block_tables;
    const int32_t *seq_lens;
    const int32_t *starts;         // [num_seqs] first position whose block changed, or null: 0
    uint32_t *err;
    int num_seqs, num_kv_heads, max_blocks, num_blocks;
};

// pa_select_blocks: the blocks whose bounds promise the largest scores.
struct SelectParams {
    int32_t *tiles;                // [num_seqs][num_kv_heads][keep]
    int32_t *tile_lens;            // [num_seqs][num_kv_heads]
    const void *q;
    const void *bounds;
    const int32_t *block_tables;
    const int32_t *seq_lens;
    uint32_t *scores;              // workspace: [num_seqs][num_kv_heads][row] fp32 scores as
                                   //   ordered numbers, if they are computed apart or do not
                                   //   fit shared memory,
    float *sizes;                  //   [..][row / 16] with those the largest sum |q||bound|,
    unsigned long long *exact;     //   [..][row] scores with more bits, of those in doubt
    uint32_t *err;
    int num_seqs, num_heads, num_kv_heads, max_blocks, num_blocks;
    int keep, keep_first, keep_last;
    int row;                       // max_blocks rounded up to 16
    int near;                      // scores a thread block holds in shared memory, or 0
};

// The selection's launch, and before it that of the scores (or null).
struct SelectLaunch {
    const void *fn, *score_fn;
    int threads, near, score_threads, score_blocks;
    size_t smem;
};

// pa_evict: a sequence shortened to its heaviest tokens.
struct EvictParams {
    void *k_cache, *v_cache;
    float *mass;                   // [num_seqs][num_kv_heads][max_blocks * 16]
    const int32_t *block_tables;
    const int32_t *seq_lens;
    const int32_t *new_lens;
    int32_t *lists;                // workspace: per (sequence, head) `list` holes, then sources
    uint32_t *err;
    int num_seqs, num_kv_heads, max_blocks, num_blocks;
    int keep_first, keep_last;
    int list;
    int keys, table;               // masses and table entries a block holds in shared memory
};

// A launch of the eviction kernel.
struct EvictLaunch {
    const void *fn;
    int threads, cluster, keys, table;
    size_t smem;
};

struct SparseKernel {
    const void *fn;
    int threads;
};

SparseKernel bounds_kernel(bool bf16, int head_dim);
SelectLaunch select_launch(bool bf16, int head_dim, int group, int num_runs, int max_blocks,
                           int keep, int num_sms);
EvictLaunch evict_launch(int head_dim, int num_runs, int max_blocks, int num_sms);

}  // namespace pa
