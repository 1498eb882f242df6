// pa_select.cu -- which blocks of a long sequence a query should read
// (sm_103a): per-block bounds of the keys, and the choice of blocks by the
// scores that the bounds allow.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include "pa_device.cuh"
#include "pa_ragged.cuh"
#include "pa_sparse.h"

namespace pa {

namespace {

template <typename T>
struct Pair;
template <>
struct Pair<__half> {
    using V = __half2;
};
template <>
struct Pair<__nv_bfloat16> {
    using V = __nv_bfloat162;
};

// min and max of two pairs of 16-bit values; a NaN wins
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
{
    using V = typename Pair<T>::V;
    const V r = __hmin2_nan(*reinterpret_cast<V *>(&a), *reinterpret_cast<V *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    using V = typename Pair<T>::V;
    const V r = __hmax2_nan(*reinterpret_cast<V *>(&a), *reinterpret_cast<V *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// the larger of two pairs of magnitudes; a NaN loses
template <typename T>
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b)
{
    using V = typename Pair<T>::V;
    const V r = __hmax2(*reinterpret_cast<V *>(&a), *reinterpret_cast<V *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

constexpr int kBoundsThreads = 256;

// ---------------------------------------------------------------------------
// bounds[b][h][0][c] = min_t k[b][h][t][c], bounds[b][h][1][c] = max_t, over the
// block's live tokens.  One warp takes a (block, kv head) tile: all of its
// 16-byte loads (8 a lane at head_dim 128) are in flight at once, the rows meet
// in packed 16-bit minima and maxima and one or two shuffles, and half of
// the lanes write the minima, half the maxima.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kBoundsThreads) block_bounds_kernel(const BoundsParams p)
{
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int CPR = D / 8;                    // 16-byte chunks of a row
    constexpr int RPL = 32 / CPR;                 // rows a warp loads at once
    constexpr int NL = kBlockSize / RPL;
    __shared__ RaggedSmem sm;
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kBoundsThreads / 32);
    const int me = blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5);
    const int Hkv = p.num_kv_heads;
    const int ch = lane % CPR, rr = lane / CPR;
    grid_dependents_launch();
    grid_dependency_wait();
    // the first block of sequence s that changed, and how many there are
    auto first_of = [&](int s, int L) {
        const int b = p.starts ? __ldg(p.starts + s) : 0;
        return min(max(b, 0), L) / kBlockSize;
    };
    for (int begin = 0; begin < p.num_seqs; begin += kRaggedSeqs) {
        const int n = min(kRaggedSeqs, p.num_seqs - begin);
        ragged_prefix<kBoundsThreads>(sm, begin, n, [&](int s) {
            const int L = checked_len(p.seq_lens, s, p.max_blocks, p.err);
            if (p.starts) {
                const int b = __ldg(p.starts + s);
                if (b < 0 || b > L)
                    record_error(p.err, PA_DEVERR_QUERY_RANGE);
                if (b >= L)
                    return 0;
            }
            return (L + kBlockSize - 1) / kBlockSize - first_of(s, L);
        });
        // heads of a block lie one after the other: unit = block * Hkv + head
        const long long total = (long long)sm.pre[n] * Hkv;
        const long long share = (total + warps - 1) / warps;
        long long u = me * share;
        const long long end = min(total, u + share);
        if (u >= end)
            continue;
        int i = ragged_find(sm, n, (int)(u / Hkv));
        int j = (int)(u / Hkv), h = (int)(u % Hkv);
        while (u < end) {
            while (j >= sm.pre[i + 1])
                ++i;
            const int s = begin + i;
            const int L = min(max(__ldg(p.seq_lens + s), 0), p.max_blocks * kBlockSize);
            const int b = first_of(s, L) + j - sm.pre[i];
            const int phys = __ldg(p.block_tables + (size_t)s * p.max_blocks + b);
            if ((unsigned)phys < (unsigned)p.num_blocks) {
                const int last = min(kBlockSize, L - b * kBlockSize) - 1;
                const size_t tile = (size_t)phys * Hkv + h;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const T *>(p.k_cache) + tile * kBlockSize * D);
                uint4 x[NL];
#pragma unroll
                for (int l = 0; l < NL; ++l)      // rows past the last live one: that one again
                    x[l] = __ldcs(src + min(l * RPL + rr, last) * CPR + ch);
                uint4 lo = x[0], hi = x[0];
#pragma unroll
                for (int l = 1; l < NL; ++l) {
                    lo.x = min2<T>(lo.x, x[l].x), hi.x = max2<T>(hi.x, x[l].x);
                    lo.y = min2<T>(lo.y, x[l].y), hi.y = max2<T>(hi.y, x[l].y);
                    lo.z = min2<T>(lo.z, x[l].z), hi.z = max2<T>(hi.z, x[l].z);
                    lo.w = min2<T>(lo.w, x[l].w), hi.w = max2<T>(hi.w, x[l].w);
                }
#pragma unroll
                for (int off = CPR; off < 32; off <<= 1) {
                    lo.x = min2<T>(lo.x, __shfl_xor_sync(FULL, lo.x, off));
                    lo.y = min2<T>(lo.y, __shfl_xor_sync(FULL, lo.y, off));
                    lo.z = min2<T>(lo.z, __shfl_xor_sync(FULL, lo.z, off));
                    lo.w = min2<T>(lo.w, __shfl_xor_sync(FULL, lo.w, off));
                    hi.x = max2<T>(hi.x, __shfl_xor_sync(FULL, hi.x, off));
                    hi.y = max2<T>(hi.y, __shfl_xor_sync(FULL, hi.y, off));
                    hi.z = max2<T>(hi.z, __shfl_xor_sync(FULL, hi.z, off));
                    hi.w = max2<T>(hi.w, __shfl_xor_sync(FULL, hi.w, off));
                }
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.bounds) + tile * 2 * D);
                if (rr < 2)
                    dst[rr * CPR + ch] = rr ? hi : lo;
            } else if (lane == 0) {
                record_error(p.err, PA_DEVERR_TABLE_RANGE);
            }
            ++u;
            if (++h == Hkv) {
                h = 0;
                ++j;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The score of a block is the largest q.k that its bounds allow, the greatest
// of the group's heads:
//     score_j = max_g sum_c max(q_gc min_jc, q_gc max_jc)
//             = max_g (max(q_g, 0) . max_j + min(q_g, 0) . min_j),
// a matrix product over 2 head_dim channels.  A warp takes 16 blocks (rows of
// the A operand), the group's heads are the columns.  The channels of a product
// may be taken in any order, so a lane loads 16 bytes of a row at a time
// straight into its fragments (8 neighbouring channels, as two k-steps of four)
// and the queries are laid out to match; no shared memory.
// ---------------------------------------------------------------------------
constexpr int kScoreThreads = 128;

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kScoreThreads) block_score_kernel_t(const SelectParams p)
{
    using M = Mma<T>;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int NI = D / 32;                    // 16-byte loads of a row's minima (maxima)
    __shared__ RaggedSmem sm;
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kScoreThreads / 32);
    const int me = blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv;
    const int r = lane >> 2, qd = lane & 3;
    grid_dependents_launch();
    grid_dependency_wait();
    for (int begin = 0; begin < p.num_seqs; begin += kRaggedSeqs) {
        const int n = min(kRaggedSeqs, p.num_seqs - begin);
        ragged_prefix<kScoreThreads>(sm, begin, n, [&](int s) {
            const int L = checked_len(p.seq_lens, s, p.max_blocks, p.err);
            const int nb = (L + kBlockSize - 1) / kBlockSize;
            return nb <= p.keep ? 0 : (nb + 15) / 16;   // all are kept: no scores wanted
        });
        const long long total = (long long)sm.pre[n] * Hkv;
        const long long share = (total + warps - 1) / warps;
        long long u = me * share;
        const long long end = min(total, u + share);
        if (u >= end)
            continue;
        int i = ragged_find(sm, n, (int)(u / Hkv));
        int nt = sm.pre[i + 1] - sm.pre[i];
        int h = (int)((u - (long long)sm.pre[i] * Hkv) / nt);
        int t = (int)((u - (long long)sm.pre[i] * Hkv) % nt);
        bool fresh = true;
        uint32_t qn[NT][NI][4], qp[NT][NI][4];    // min(q, 0) and max(q, 0)
        int nb = 0;
        for (; u < end; ++u) {
            const int s = begin + i;
            if (fresh) {
                fresh = false;
                const int L = min(max(__ldg(p.seq_lens + s), 0), p.max_blocks * kBlockSize);
                nb = (L + kBlockSize - 1) / kBlockSize;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int g = 8 * j + r;
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        static_cast<const T *>(p.q) +
                        ((size_t)s * p.num_heads + h * G + min(g, G - 1)) * D);
#pragma unroll
                    for (int k = 0; k < NI; ++k) {
                        const uint4 x = __ldg(src + 4 * k + qd);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            qn[j][k][e] = min2<T>(w[e], 0u);
                            qp[j][k][e] = max2<T>(w[e], 0u);
                        }
                    }
                }
            }
            // rows r and r + 8 of the 16 blocks; past the end the last block again
            const int32_t *table = p.block_tables + (size_t)s * p.max_blocks;
            const uint4 *row[2];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                int phys = __ldg(table + min(16 * t + 8 * a + r, nb - 1));
                if ((unsigned)phys >= (unsigned)p.num_blocks) {
                    record_error(p.err, PA_DEVERR_TABLE_RANGE);
                    phys = 0;
                }
                row[a] = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.bounds) +
                                                         ((size_t)phys * Hkv + h) * 2 * D) + qd;
            }
            uint4 x[2][2 * NI];
#pragma unroll
            for (int k = 0; k < 2 * NI; ++k)
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    x[a][k] = __ldg(row[a] + 4 * k);
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
            uint32_t big = 0;
#pragma unroll
            for (int k = 0; k < 2 * NI; ++k) {
                const uint32_t a0[4] = {x[0][k].x, x[1][k].x, x[0][k].y, x[1][k].y};
                const uint32_t a1[4] = {x[0][k].z, x[1][k].z, x[0][k].w, x[1][k].w};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint32_t *q = k < NI ? qn[j][k] : qp[j][k - NI];
                    M::run(acc[j], a0, q[0], q[1]);
                    M::run(acc[j], a1, q[2], q[3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    big = most2<T>(big, a0[e] & 0x7fff7fffu);
                    big = most2<T>(big, a1[e] & 0x7fff7fffu);
                }
            }
            // the greatest head's score of block r (and r + 8); not finite: first of all
            float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = fabsf(acc[j][e]) <= FLT_MAX ? acc[j][e] : INFINITY;
                    if (8 * j + 2 * qd + (e & 1) < G)
                        best[e >> 1] = fmaxf(best[e >> 1], v);
                }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                best[0] = fmaxf(best[0], __shfl_xor_sync(FULL, best[0], off));
                best[1] = fmaxf(best[1], __shfl_xor_sync(FULL, best[1], off));
            }
            const float2 b2 = Elem<T>::to_f2(big);
            float reach = fmaxf(b2.x, b2.y);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1)
                reach = fmaxf(reach, __shfl_xor_sync(FULL, reach, off));
            const size_t out = ((size_t)s * Hkv + h) * p.row + 16 * t;
            if (qd < 2 && 16 * t + 8 * qd + r < nb)
                p.scores[out + 8 * qd + r] = best[qd];
            if (lane == 0)
                p.reach[out / 16] = reach;
            if (++t == nt) {
                t = 0;
                fresh = true;
                if (++h == Hkv) {
                    h = 0;
                    do
                        ++i;
                    while (i < n && sm.pre[i + 1] == sm.pre[i]);
                    if (i < n)
                        nt = sm.pre[i + 1] - sm.pre[i];
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The choice: per (sequence, kv head) the keep_first first blocks, the keep_last
// last ones and the best of the rest.  The tensor cores' sums are off by a part
// of sum |q||bound|, and the choice must not depend on that: with E the largest
// error, a block whose score lies more than 2 E above the lowest chosen one is
// in, one that lies more than 2 E below is out, and the few between are
// summed again in pairs of floats (46 bits) and ranked by that, ties to the lowest
// position.
// ---------------------------------------------------------------------------
constexpr int kSelectThreads = 512;
constexpr int kSelectBins = 2048;
constexpr int kDoubt = 512;                       // blocks in doubt that are ranked directly

// The order of floats as unsigned numbers (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// (s, e) += x without loss of what falls off s
__device__ __forceinline__ void two_add(float &s, float &e, float x)
{
    const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
    e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
}

template <typename T, int D>
__global__ void __launch_bounds__(kSelectThreads) block_select_kernel_t(const SelectParams p)
{
    constexpr int NTH = kSelectThreads, NW = NTH / 32;
    constexpr uint32_t FULL = 0xffffffffu;
    __shared__ float q[kMaxGroup * D];            // the group's queries
    __shared__ int hist[kSelectBins];
    __shared__ int doubt[kDoubt];
    __shared__ unsigned long long key[kDoubt];
    __shared__ float red[3][NW];
    __shared__ int redi[2][NW];
    __shared__ int count[2];                      // blocks in doubt, and above them
    __shared__ int found;                         // the lowest chosen one's bin
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv;
    const int run = blockIdx.x, s = run / Hkv, h = run % Hkv;
    grid_dependents_launch();
    grid_dependency_wait();
    int L = __ldg(p.seq_lens + s);
    if (L < 0 || L > p.max_blocks * kBlockSize) {
        if (tid == 0)
            record_error(p.err, PA_DEVERR_SEQLEN_RANGE);
        L = L < 0 ? 0 : p.max_blocks * kBlockSize;
    }
    const int nb = (L + kBlockSize - 1) / kBlockSize;
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks;
    int32_t *out = p.tiles + (size_t)run * p.keep;
    auto tile_of = [&](int j) {
        const int phys = __ldg(table + j);
        if ((unsigned)phys >= (unsigned)p.num_blocks) {
            record_error(p.err, PA_DEVERR_TABLE_RANGE);
            return h;                             // block 0's tile, as the score was taken
        }
        return phys * Hkv + h;
    };
    if (tid == 0)
        p.tile_lens[run] = L - kBlockSize * max(0, nb - p.keep);
    if (nb <= p.keep) {
        for (int j = tid; j < p.keep; j += NTH)
            out[j] = j < nb ? tile_of(j) : -1;
        return;
    }
    const int lo = p.keep_first, hi = nb - p.keep_last;   // the blocks that compete
    int want = p.keep - p.keep_first - p.keep_last;       // how many of them are kept
    float *score = p.scores + (size_t)run * p.row;
    const float *reach = p.reach + (size_t)run * (p.row / 16);

    // queries, their largest sum of magnitudes, the largest |bound|, the scores' range
    for (int i = tid; i < G * D; i += NTH)
        q[i] = Elem<T>::to_f(static_cast<const T *>(p.q)[((size_t)s * p.num_heads + h * G) * D + i]);
    for (int i = tid; i < kSelectBins; i += NTH)
        hist[i] = 0;
    if (tid < 2)
        count[tid] = 0;
    __syncthreads();
    float most = 0.f, least_s = INFINITY, most_s = -INFINITY;
    int first_of_all = 0;                         // scores that are not finite
    for (int i = tid; i < (nb + 15) / 16; i += NTH)
        most = fmaxf(most, __ldcg(reach + i));
    for (int j = lo + tid; j < hi; j += NTH) {
        const float x = __ldcg(score + j);
        if (x == INFINITY) {
            ++first_of_all;
        } else {
            least_s = fminf(least_s, x);
            most_s = fmaxf(most_s, x);
        }
    }
    float l1 = 0.f;
    for (int g = warp; g < G; g += NW) {
        float a = 0.f;
        for (int c = lane; c < D; c += 32)
            a += fabsf(q[g * D + c]);
#pragma unroll
        for (int off = 16; off; off >>= 1)
            a += __shfl_xor_sync(FULL, a, off);
        l1 = fmaxf(l1, a);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        most = fmaxf(most, __shfl_xor_sync(FULL, most, off));
        least_s = fminf(least_s, __shfl_xor_sync(FULL, least_s, off));
        most_s = fmaxf(most_s, __shfl_xor_sync(FULL, most_s, off));
    }
    first_of_all = __reduce_add_sync(FULL, first_of_all);
    if (lane == 0) {
        red[0][warp] = most;
        red[1][warp] = least_s;
        red[2][warp] = most_s;
        redi[0][warp] = first_of_all;
        redi[1][warp] = __float_as_int(l1);       // not negative: ordered as an int
    }
    __syncthreads();
    first_of_all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        most = fmaxf(most, red[0][w]);
        least_s = fminf(least_s, red[1][w]);
        most_s = fmaxf(most_s, red[2][w]);
        first_of_all += redi[0][w];
        l1 = fmaxf(l1, __int_as_float(redi[1][w]));
    }
    // Largest error: 2 D / 16 steps each add 17 terms aligned to the largest, none above
    // sum |q||bound| <= l1 * most, and lose 2^-23 of it a term
    // (infinite bounds put everything in doubt)
    const float twice = 2.f * (2 * D / 16) * 17 * 1.1920929e-7f * l1 * most;
    const float slack = twice <= FLT_MAX ? twice : FLT_MAX;
    // scores that are not finite rank first: all of them, or the foremost
    int inf_left = min(first_of_all, want);
    want -= inf_left;
    // bins of equal width over the finite scores; the bin rises with the score
    const float width = (most_s - least_s) / kSelectBins;
    const float per = width > 0.f ? 1.f / width : 0.f;
    auto bin_of = [&](float x) {
        const float b = (x - least_s) * per;
        return b >= (float)(kSelectBins - 1) ? kSelectBins - 1 : b > 0.f ? (int)b : 0;
    };
    int cut = kSelectBins;                        // no bin lies above: none is kept
    if (want > 0) {
        for (int j = lo + tid; j < hi; j += NTH) {
            const float x = __ldcg(score + j);
            if (x != INFINITY)
                atomicAdd(&hist[bin_of(x)], 1);
        }
        __syncthreads();
        // the bin of the want-th largest: each thread sums its bins, the warps' sums are
        // scanned from the top
        constexpr int BPT = kSelectBins / NTH;
        int mine = 0;
#pragma unroll
        for (int b = 0; b < BPT; ++b)
            mine += hist[kSelectBins - 1 - (tid * BPT + b)];
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, incl, o);
            if (lane >= o)
                incl += y;
        }
        if (lane == 31)
            redi[0][warp] = incl;
        __syncthreads();
        int above = incl - mine;
        for (int w = 0; w < warp; ++w)
            above += redi[0][w];
        if (above < want && above + mine >= want) {
            int b = 0;
            for (; b < BPT - 1 && above + hist[kSelectBins - 1 - (tid * BPT + b)] < want; ++b)
                above += hist[kSelectBins - 1 - (tid * BPT + b)];
            found = kSelectBins - 1 - (tid * BPT + b);
        }
        __syncthreads();
        cut = found;
        // in, out, or in doubt
        int sure = 0;
        for (int j = lo + tid; j < hi; j += NTH) {
            const float x = __ldcg(score + j);
            if (x == INFINITY)
                continue;
            if (bin_of(x - slack) > cut) {
                ++sure;
            } else if (bin_of(x + slack) >= cut) {
                const int at = atomicAdd(&count[0], 1);
                if (at < kDoubt)
                    doubt[at] = j;
            }
        }
        sure = __reduce_add_sync(FULL, sure);
        if (lane == 0 && sure)
            atomicAdd(&count[1], sure);
        __syncthreads();
        const int need = want - count[1];
        const int c = count[0];
        // the score of block j by the warp, as an ordered number of 64 bits
        auto resum = [&](int j) {
            const int phys = __ldg(table + j);
            const T *b = static_cast<const T *>(p.bounds) +
                         ((size_t)((unsigned)phys < (unsigned)p.num_blocks ? phys : 0) * Hkv + h) *
                             2 * D;
            unsigned long long best = 0;
            for (int g = 0; g < G; ++g) {
                float a = 0.f, e = 0.f;
#pragma unroll
                for (int cc = 0; cc < D; cc += 32) {
                    const float qc = q[g * D + cc + lane];
                    const float k = Elem<T>::to_f(b[(qc > 0.f ? D : 0) + cc + lane]);
                    two_add(a, e, qc * k);        // an exact product
                }
#pragma unroll
                for (int off = 16; off; off >>= 1) {
                    const float oa = __shfl_xor_sync(FULL, a, off);
                    const float oe = __shfl_xor_sync(FULL, e, off);
                    two_add(a, e, oa);
                    e += oe;
                }
                const float x = __fadd_rn(a, e), rest = __fsub_rn(e, __fsub_rn(x, a));
                const unsigned long long kk =
                    (unsigned long long)ordered(x) << 32 | ordered(rest);
                best = kk > best ? kk : best;
            }
            return __shfl_sync(FULL, best, 0);
        };
        if (c <= kDoubt) {
            for (int i = warp; i < c; i += NW) {
                const unsigned long long k = resum(doubt[i]);
                if (lane == 0)
                    key[i] = k;
            }
            __syncthreads();
            for (int i = tid; i < c; i += NTH) {
                const unsigned long long k = key[i];
                const int j = doubt[i];
                int better = 0;
                for (int o = 0; o < c; ++o)
                    better += key[o] > k || (key[o] == k && doubt[o] < j);
                // what is in stands at the top of its bins from here on, what is out at the bottom
                score[j] = better < need ? FLT_MAX : -FLT_MAX;
            }
        } else {
            // very many scores close together (equal blocks): the need-th largest key bit
            // by bit
            unsigned long long *keys = p.exact + (size_t)run * p.row;
            auto doubtful = [&](float x) {
                return x != INFINITY && bin_of(x - slack) <= cut && bin_of(x + slack) >= cut;
            };
            for (int j = lo + warp; j < hi; j += NW) {
                unsigned long long k = 0;
                if (doubtful(__ldcg(score + j)))
                    k = resum(j);
                if (lane == 0)
                    keys[j] = k;
            }
            __syncthreads();
            unsigned long long edge = 0;
            auto tally = [&](unsigned long long at_least) {
                int m = 0;
                for (int j = lo + tid; j < hi; j += NTH)
                    m += __ldcg(keys + j) >= at_least;
                m = __reduce_add_sync(FULL, m);
                if (lane == 0)
                    redi[1][warp] = m;
                __syncthreads();
                m = 0;
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    m += redi[1][w];
                __syncthreads();
                return m;
            };
            for (int bit = 63; bit >= 0; --bit)
                if (tally(edge | 1ull << bit) >= need)
                    edge |= 1ull << bit;
            // of those at the edge the first ones
            int left = need - tally(edge + 1);
            for (int base = lo; base < hi; base += NTH) {
                const int j = base + tid;
                const unsigned long long k = j < hi ? __ldcg(keys + j) : 0;
                const bool tie = j < hi && k == edge;
                const unsigned ballot = __ballot_sync(FULL, tie);
                if (lane == 0)
                    redi[1][warp] = __popc(ballot);
                __syncthreads();
                int before = 0, all = 0;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    before += w < warp ? redi[1][w] : 0;
                    all += redi[1][w];
                }
                if (j < hi && k)
                    score[j] = k > edge || (tie && before + __popc(ballot & ((1u << lane) - 1)) < left)
                                   ? FLT_MAX
                                   : -FLT_MAX;
                left -= min(left, all);
                __syncthreads();
            }
        }
    }
    __syncthreads();                              // the scores' marks
    // the kept blocks in their order
    int at = 0;
    for (int base = 0; base < nb; base += NTH) {
        const int j = base + tid;
        bool in = false, inf = false;
        if (j < nb) {
            if (j < lo || j >= hi) {
                in = true;
            } else {
                const float x = __ldcg(score + j);
                inf = x == INFINITY;
                in = !inf && want > 0 && (x == FLT_MAX || (x != -FLT_MAX && bin_of(x - slack) > cut));
            }
        }
        const unsigned infb = __ballot_sync(FULL, inf);
        const unsigned inb = __ballot_sync(FULL, in);
        if (lane == 0) {
            redi[0][warp] = __popc(inb);
            redi[1][warp] = __popc(infb);
        }
        __syncthreads();
        const unsigned below = (1u << lane) - 1;
        int ins = 0, infs_before = 0, all_in = 0, all_inf = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) {
                ins += redi[0][w];
                infs_before += redi[1][w];
            }
            all_in += redi[0][w];
            all_inf += redi[1][w];
        }
        ins += __popc(inb & below);
        infs_before += __popc(infb & below);
        if (inf)
            in = infs_before < inf_left;
        if (in)
            out[at + ins + min(infs_before, inf_left)] = tile_of(j);
        at += all_in + min(all_inf, inf_left);
        inf_left -= min(all_inf, inf_left);
        __syncthreads();
    }
}

}  // namespace

SparseKernel bounds_kernel(bool bf16, int head_dim)
{
    SparseKernel k{nullptr, kBoundsThreads};
    if (head_dim == 128)
        k.fn = bf16 ? reinterpret_cast<const void *>(&block_bounds_kernel<__nv_bfloat16, 128>)
                    : reinterpret_cast<const void *>(&block_bounds_kernel<__half, 128>);
    else
        k.fn = bf16 ? reinterpret_cast<const void *>(&block_bounds_kernel<__nv_bfloat16, 64>)
                    : reinterpret_cast<const void *>(&block_bounds_kernel<__half, 64>);
    return k;
}

template <typename T, int D>
static const void *score_fn(int group)
{
    return group <= 8 ? reinterpret_cast<const void *>(&block_score_kernel_t<T, D, 1>)
                      : reinterpret_cast<const void *>(&block_score_kernel_t<T, D, 2>);
}

SparseKernel block_score_kernel(bool bf16, int head_dim, int group)
{
    SparseKernel k{nullptr, kScoreThreads};
    if (head_dim == 128)
        k.fn = bf16 ? score_fn<__nv_bfloat16, 128>(group) : score_fn<__half, 128>(group);
    else
        k.fn = bf16 ? score_fn<__nv_bfloat16, 64>(group) : score_fn<__half, 64>(group);
    return k;
}

SparseKernel block_select_kernel(bool bf16, int head_dim)
{
    SparseKernel k{nullptr, kSelectThreads};
    if (head_dim == 128)
        k.fn = bf16 ? reinterpret_cast<const void *>(&block_select_kernel_t<__nv_bfloat16, 128>)
                    : reinterpret_cast<const void *>(&block_select_kernel_t<__half, 128>);
    else
        k.fn = bf16 ? reinterpret_cast<const void *>(&block_select_kernel_t<__nv_bfloat16, 64>)
                    : reinterpret_cast<const void *>(&block_select_kernel_t<__half, 64>);
    return k;
}

}  // namespace pa
