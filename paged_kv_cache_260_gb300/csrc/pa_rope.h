// pa_rope.h -- what the host side of pa_rope_and_cache and pa_qk_norm_rope
// shares with their kernel (pa_rope.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pa {

struct RopeParams {
    const void *q, *k, *v;         // rows of num_heads (num_kv_heads) heads, token strides below
    void *q_out;
    void *k_out;                   // without slots: the keys' rows; else null
    void *k_cache, *v_cache;       // with slots: the pools
    const int64_t *slots;          // [num_tokens], <0 = padding; null: no pool
    const int32_t *positions;      // [num_tokens], <0 = padding
    const float *cos_sin;          // [max_position][rotary_dim]: cosines, then sines
    const void *q_norm, *k_norm;   // [head_dim / num_maps] weights, or null: not normalised
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // elements a token
    long long num_slots;
    uint32_t *err;
    int num_tokens;
    int num_kv_heads;
    int num_maps;                  // equal parts of a head that are normalised and rotated apart
    int q_segs, k_segs, v_segs;    // parts of a token's q, k and v rows (v_segs 0 without a pool)
    int rotary_dim, max_position;
    float eps;
};

// How many units are handed out: the first long_blocks blocks share the first
// long_units evenly, the blocks after them take short_units each.
struct RopeSplit {
    unsigned long_blocks, long_units, short_units;
};

// A launch with arguments (RopeParams, int iters, and for the kernel with
// dynamic shared memory RopeSplit).
struct RopeKernel {
    const void *fn;
    int threads, blocks;
    size_t smem;                   // dynamic shared memory a block
    int iters;                     // rounds of segments in a unit of work
    RopeSplit split;
};

// The kernel and its grid for one call; fn is null if the call has more units
// of work than it can count.
RopeKernel rope_kernel(const RopeParams &p, bool bf16, int head_dim, bool interleaved, int num_sms);

}  // namespace pa
