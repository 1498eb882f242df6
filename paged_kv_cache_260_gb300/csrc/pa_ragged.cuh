// pa_ragged.cuh -- equal shares of a ragged batch: units of work that each
// sequence has a number of, handed to the warps of a grid.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

struct RaggedSmem {
    int32_t pre[kRaggedSeqs + 1];  // units of the part's sequences before this one
    int32_t warp_sum[32];
};

// Fill pre for sequences [begin, begin + n), n <= kRaggedSeqs, count(s) units
// each; every thread of the block calls it.  The counts of a part stay below 2^31.
template <int NT, typename F>
__device__ __forceinline__ void ragged_prefix(RaggedSmem &sm, int begin, int n, const F &count)
{
    constexpr int K = kRaggedSeqs / NT;
    constexpr uint32_t FULL = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __syncthreads();                              // the part before has been walked
    int carry = 0;
    // K rows of NT neighbouring sequences; a batch of a few rows walks only those
    for (int row = 0; row < K && row * NT < n; ++row) {
        const int i = row * NT + tid;
        const int c = i < n ? count(begin + i) : 0;
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, incl, o);
            if (lane >= o)
                incl += y;
        }
        if (lane == 31)
            sm.warp_sum[warp] = incl;
        __syncthreads();
        int before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            const int x = sm.warp_sum[w];
            before += w < warp ? x : 0;
            total += x;
        }
        if (i < n)
            sm.pre[i] = carry + before + incl - c;
        carry += total;
        __syncthreads();                          // warp_sum is reused
    }
    if (tid == 0)
        sm.pre[n] = carry;
    __syncthreads();
}

// largest i with pre[i] <= u (sequences without units are skipped)
__device__ __forceinline__ int ragged_find(const RaggedSmem &sm, int n, int u)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sm.pre[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// A length as the kernels use it: out of [0, max_blocks * 16] is clamped and reported.
__device__ __forceinline__ int checked_len(const int32_t *seq_lens, int s, int max_blocks,
                                           uint32_t *err)
{
    const int L = __ldg(seq_lens + s);
    if (L < 0 || L > max_blocks * kBlockSize) {
        record_error(err, PA_DEVERR_SEQLEN_RANGE);
        return L < 0 ? 0 : max_blocks * kBlockSize;
    }
    return L;
}

}  // namespace pa
