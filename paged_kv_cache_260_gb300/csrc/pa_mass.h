// pa_mass.h -- what the host side of pa_decode_mass and pa_prefill_mass shares
// with the kernels that add up softmax weights per token.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pa {

// The accounting after a decode: scores and statistics of DecodeParams.
struct DecodeMassParams {
    float *mass;                   // [num_seqs][num_kv_heads][max_blocks * 16]
    const float *scores;           // [num_seqs * num_kv_heads][max_blocks * 16][score_cols]
    const float2 *stat;            // [num_seqs][num_heads] maximum (base 2), 1 / sum
    const int32_t *seq_lens;
    int num_seqs, num_heads, num_kv_heads, max_blocks;
    float decay;
};

// The weights a chunk's queries give: two passes over the keys and a sum.
struct PrefillMassParams {
    float *mass;
    const void *q, *k_cache;
    const int32_t *block_tables;
    const int32_t *seq_lens;
    const int32_t *query_start;
    float2 *stats;                 // [unit + block][2 halves][2 * 128 rows] maximum (base 2),
                                   // sum
    float *sums;                   // [num_seqs * num_kv_heads][2 * row_blocks][max_blocks * 16]
    uint32_t *err;
    int num_seqs, num_heads, num_kv_heads, max_blocks, num_blocks;
    int num_queries;               // rows of q
    // units of 2 x 128 (token, head) rows per (sequence, kv head): a launch takes row_blocks of
    // them, from block0 on, of the longest chunk's all_blocks
    int row_blocks, block0, all_blocks;
    // few rows: columns of the kept scores (in sums, [run][max_blocks * 16][columns]), the longest
    // chunk, the first kernel's warps; stats are [run + warp][kMassFewRows]
    int few_cols, few_tokens, few_warps;
    float scale_log2, decay;
};

// Sums or scores that pa_prefill_mass keeps at a time, a gigabyte of workspace, and scores that
// pa_decode_mass does, four.  What would be more is taken in parts (but for one sequence's or
// one row block's own).  A part of a chunk's row blocks is milliseconds long where the tables
// are full; one of a decode costs 10 us: 128 sequences of the lognormal lengths to 4096 in tables
// for 131K tokens, 2.2 GB in one part, 88.3 us in a graph, 98.2 in two; of eight times the
// lengths 647 and 669.
constexpr long long kMassKept = 1 << 28, kMassDecodeKept = 1 << 30;

constexpr int kMassRows = 128;     // (token, head) rows of one query tile
constexpr int kMassTiles = 2;      // query tiles of a unit
constexpr int kMassKeys = 128;     // keys of a tile

// A batch whose tables hold at most kMassShortKeys tokens, and whose longest chunk's rows
// make at most kMassShortWork multiplications with them, takes the one-launch kernel: 32
// keys of 16 rows of 128 channels a warp.  Several row blocks cost the passes a third launch,
// and more is worth it.  In us in a graph, bf16, one launch / the passes, for rows (tokens x
// heads of a group) and keys, 32 runs of 128 channels: 4 x 512 10.3 / 11.0, 64 x 128 9.1 / 10.1,
// 128 x 128 13.4 / 10.1, 64 x 256 13.6 / 10.1, 512 x 128 24.1 / 15.8; 4 runs of 64 channels:
// 16 x 64 6.1 / 9.1, 4 x 512 8.2 / 9.5, 64 x 128 7.0 / 9.4, 128 x 128 9.9 / 9.2, 256 x 64
// 7.9 / 10.8, 280 x 128 16.8 / 14.1.  The tables' width is all that the host knows of the keys:
// chunks of 5 and of 70 tokens of four heads in tables of 160 keys, the long one over 70 keys
// 10.3 / 13.4, over 150 17.9 / 13.3.
constexpr int kMassShortKeys = 512;
constexpr long long kMassShortWork = 1 << 20, kMassShortWorkOfBlocks = 3 << 20;
constexpr int kMassShortThreads = 512;

// Chunks of at most this many (token, head) rows a kv head keep their scores (4 bytes a row
// and key beside 2 head_dim).  us in a graph, kept scores / the passes, 8 kv heads x 128: 8 x 16K
// keys 4 rows 57 / 108, 8 rows 63 / 108, 16 rows 79 / 109 (32 would write as many bytes as they
// read); 4 x 2048 keys 4 rows 10.1 / 18.0, 16 rows 12.6 / 18.1.  Against the one launch: 512
// runs of 512 keys 16.7 / 38.5, of 32 keys 10.8 / 24.9; up to an SM's run it is as fast or
// faster: 32 runs of 128 keys 7.8 / 8.8, of 32 keys 7.4 / 6.9, 128 runs of 128 keys 9.7 / 8.8, 16
// rows of 512 keys 13.6 / 10.3.
constexpr int kMassFewRows = 16;
constexpr int kMassFewThreads = 128;

struct MassKernels {
    const void *stats, *sums;      // (PrefillMassParams, tensor map of the key pool)
    const void *whole;             // (PrefillMassParams): short sequences
    const void *few[2], *few_finish;       // (PrefillMassParams): up to 8 and 16 rows
    int threads;
    size_t smem_stats, smem_sums;
};

bool prefill_mass_kernels(bool bf16, int head_dim, MassKernels *k);
const void *prefill_mass_finish();     // (PrefillMassParams)
const void *decode_mass_finish();      // (DecodeMassParams)
constexpr int kMassFinishThreads = 256;

}  // namespace pa
