// pa_select.cu -- which blocks of a long sequence a query should read
// (sm_103a): per-block bounds of the keys, and the choice of blocks by the
// scores that the bounds allow.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include "pa_device.cuh"
#include "pa_ragged.cuh"
#include "pa_sparse.h"
#include "pa_tally.cuh"

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

constexpr int kBoundsThreads = 256;

// ---------------------------------------------------------------------------
// bounds[b][h][0][c] = min_t k[b][h][t][c], bounds[b][h][1][c] = max_t, over the
// block's live tokens.  One warp takes a (block, kv head) tile: all of its
// 16-byte loads (8 a lane at head_dim 128) are in flight at once, the rows meet
// in packed 16-bit minima and maxima and one or two shuffles, and half of
// the lanes write the minima, half the maxima.  HBM bounds it: 16 prompts of 16K tokens, 8
// heads x 128, 604 MB in 100 us (6.0 TB/s; five blocks an SM is what 48 registers leave).  A
// decode step's 1024 tiles are one round of loads: 3.9 us in a graph, the launch's time.
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
                // (the newest token of a sequence that has none is at -1)
                if ((b < 0 && (L > 0 || b < -1)) || b > L)
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
// The choice of blocks.  The score of a block is the largest q.k that its
// bounds allow, the greatest of the group's heads:
//     score_j = max_g sum_c max(q_gc min_jc, q_gc max_jc)
//             = max_g (max(q_g, 0) . max_j + min(q_g, 0) . min_j),
// a matrix product over 2 head_dim channels.  A warp takes 16 blocks (rows of
// the A operand), the group's heads are the columns.  The channels of a product
// may be taken in any order, so a lane loads 16 bytes of a row at a time
// straight into its fragments (8 neighbouring channels, as two k-steps of four)
// and the queries are laid out to match.
//
// Per (sequence, kv head) the keep_first first blocks, the keep_last last ones and
// the best of the rest are kept.  The tensor cores' sums are off by a part of
// sum |q||bound|, and the choice must not depend on that.  With E the largest
// error and t above the best score left out and not above the lowest one chosen,
// a block whose score lies above t + 2 E is in (its exact score is larger than
// those of all left out), one below t - 2 E is out, and the few between are
// summed again in pairs of floats (46 bits) and ranked by that, ties to the
// lowest position.  (Where scores are equal at the border, t is that score, and
// all of them lie between.)
//
// One thread block takes a (sequence, kv head), computes its scores and keeps them in
// shared memory (in the workspace, where they are more than p.near).  Few long
// sequences would leave most SMs idle: their scores are computed first, by a
// kernel whose warps share out all of them evenly, and read from the workspace
// (SCORED).
//
// The bounds are read once, 4 head_dim bytes a block and kv head.  With many runs HBM
// bounds the scores and a block's choice comes after its own: 1024 runs to 16K tokens, 278 MB,
// 70 us cold (60 % of the copy rate).  With few runs the scores of 4 x 32K to 131K tokens, 84
// MB, take 16 us from L2 and 20 from HBM, and the choice of 256 of 8192 blocks 9 more: a chain
// of passes over the scores in shared memory, a barrier each.
// ---------------------------------------------------------------------------
constexpr int kDoubt = 256;                       // blocks in doubt that are ranked directly
constexpr int kSelectNear = 16384;                // scores a block holds (64 KB)

// The order of floats as unsigned numbers (-0 as 0), and back.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_ordered(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A block's score as the selection keeps it: one that is infinite above all others.
constexpr uint32_t kFirst = 0xffffffffu;
constexpr uint32_t kIn = kFirst - 1, kOut = 1;    // one that was in doubt

__device__ __forceinline__ uint32_t score_key(float x)
{
    return x == INFINITY ? kFirst : ordered(x);
}

// (s, e) += x without loss of what falls off s
__device__ __forceinline__ void two_add(float &s, float &e, float x)
{
    const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
    e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
}

// min(q, 0) and max(q, 0) of a (sequence, kv head)'s queries as fragments of the B
// operand: lane (r, qd) holds channels 32 k + 8 qd .. + 7 of heads 8 j + r.
template <typename T, int D, int NT>
struct ScoreQueries {
    static constexpr int NI = D / 32;             // 16-byte loads of a row's minima (maxima)
    uint32_t neg[NT][NI][4], pos[NT][NI][4];

    __device__ __forceinline__ void load(const T *q, int G, int r, int qd)
    {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint4 *src = reinterpret_cast<const uint4 *>(q + min(8 * j + r, G - 1) * D);
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const uint4 x = __ldg(src + 4 * k + qd);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    neg[j][k][e] = min2<T>(w[e], 0u);
                    pos[j][k][e] = max2<T>(w[e], 0u);
                }
            }
        }
    }
};

// The scores of 16 blocks by a warp: best[0] and [1] of blocks r and r + 8, the greatest
// head's, infinite where one is not finite.  size rises to the largest sum |q||bound| of
// the others.  tile: the pool tiles of blocks r and r + 8.  between() runs while the loads
// are in flight.
template <typename T, int D, int NT, typename F>
__device__ __forceinline__ void score_tile(const ScoreQueries<T, D, NT> &q, const void *bounds,
                                           const int (&tile)[2], int G, int qd, float (&best)[2],
                                           float &size, const F &between)
{
    using M = Mma<T>;
    constexpr int NI = D / 32;
    uint4 x[2][2 * NI];
#pragma unroll
    for (int k = 0; k < 2 * NI; ++k)
#pragma unroll
        for (int a = 0; a < 2; ++a)
            x[a][k] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(bounds) +
                                                            (size_t)tile[a] * 2 * D) +
                            4 * k + qd);
    between();
    // the scores, and sum |q||bound|: the same products of magnitudes
    float acc[NT][4], mag[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[j][e] = mag[j][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 2 * NI; ++k) {
        uint32_t a0[4] = {x[0][k].x, x[1][k].x, x[0][k].y, x[1][k].y};
        uint32_t a1[4] = {x[0][k].z, x[1][k].z, x[0][k].w, x[1][k].w};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t *qq = k < NI ? q.neg[j][k] : q.pos[j][k - NI];
            M::run(acc[j], a0, qq[0], qq[1]);
            M::run(acc[j], a1, qq[2], qq[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {             // -|min| and |max|
            a0[e] = k < NI ? a0[e] | 0x80008000u : a0[e] & 0x7fff7fffu;
            a1[e] = k < NI ? a1[e] | 0x80008000u : a1[e] & 0x7fff7fffu;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t *qq = k < NI ? q.neg[j][k] : q.pos[j][k - NI];
            M::run(mag[j], a0, qq[0], qq[1]);
            M::run(mag[j], a1, qq[2], qq[3]);
        }
    }
    best[0] = best[1] = -INFINITY;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool finite = fabsf(acc[j][e]) <= FLT_MAX;
            size = finite ? fmaxf(size, mag[j][e]) : size;
            const float v = finite ? acc[j][e] : INFINITY;
            if (8 * j + 2 * qd + (e & 1) < G)
                best[e >> 1] = fmaxf(best[e >> 1], v);
        }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        best[0] = fmaxf(best[0], __shfl_xor_sync(0xffffffffu, best[0], off));
        best[1] = fmaxf(best[1], __shfl_xor_sync(0xffffffffu, best[1], off));
    }
}

// Sends for the bounds of the 16 blocks after those that are being summed, to L2: the lines of
// rows r and r + 8, one a lane of the row's four.
template <typename T, int D>
__device__ __forceinline__ void prefetch_tile(const void *bounds, const int (&tile)[2], int qd)
{
    constexpr int LINES = 2 * D * (int)sizeof(T) / 128;
    if (qd < LINES)
#pragma unroll
        for (int a = 0; a < 2; ++a)
            prefetch_l2(static_cast<const T *>(bounds) + (size_t)tile[a] * 2 * D + 64 * qd);
}

// All scores of the batch to the workspace, and of every 16 the largest sum |q||bound|.
// The warps take equal shares of the list of (sequence, kv head, 16 blocks); a sequence
// that keeps all of its blocks has none in it.
constexpr int kScoreThreads = 128;

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kScoreThreads, 4) block_score_kernel_t(const SelectParams p)
{
    __shared__ RaggedSmem sm;
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kScoreThreads / 32);
    const int me = blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv;
    const int r = lane >> 2, qd = lane & 3;
    grid_dependents_launch();
    grid_dependency_wait();
    const int n = p.num_seqs;                     // (few: see select_launch)
    ragged_prefix<kScoreThreads>(sm, 0, n, [&](int s) {
        const int L = min(max(__ldg(p.seq_lens + s), 0), p.max_blocks * kBlockSize);
        const int nb = (L + kBlockSize - 1) / kBlockSize;
        return nb <= p.keep ? 0 : (nb + 15) / 16;
    });
    const long long total = (long long)sm.pre[n] * Hkv;
    const long long share = (total + warps - 1) / warps;
    long long u = me * share;
    const long long end = min(total, u + share);
    if (u >= end)
        return;
    int i = ragged_find(sm, n, (int)(u / Hkv));
    int nt = sm.pre[i + 1] - sm.pre[i];
    int h = (int)((u - (long long)sm.pre[i] * Hkv) / nt);
    int t = (int)((u - (long long)sm.pre[i] * Hkv) % nt);
    int nb = 0;
    // rows r and r + 8 of 16 blocks; past the end the last block again
    auto tiles_of = [&](int (&tile)[2]) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            int phys = __ldg(p.block_tables + (size_t)i * p.max_blocks +
                             min(16 * t + 8 * a + r, nb - 1));
            if ((unsigned)phys >= (unsigned)p.num_blocks) {
                record_error(p.err, PA_DEVERR_TABLE_RANGE);
                phys = 0;
            }
            tile[a] = phys * Hkv + h;
        }
    };
    auto enter = [&]() {
        const int L = min(max(__ldg(p.seq_lens + i), 0), p.max_blocks * kBlockSize);
        nb = (L + kBlockSize - 1) / kBlockSize;
    };
    enter();
    ScoreQueries<T, D, NT> q;
    bool fresh = true;
    int tile[2], next[2] = {0, 0};
    tiles_of(tile);
    for (; u < end; ++u) {
        const size_t run = (size_t)i * Hkv + h;
        const int first = 16 * t, blocks = nb;
        if (fresh)
            q.load(static_cast<const T *>(p.q) + run * G * D, G, r, qd);
        fresh = false;
        float best[2], size = 0.f;
        score_tile<T, D, NT>(q, p.bounds, tile, G, qd, best, size, [&]() {
            if (++t == nt) {
                t = 0;
                fresh = true;
                if (++h == Hkv) {
                    h = 0;
                    do
                        ++i;
                    while (i < n && sm.pre[i + 1] == sm.pre[i]);
                    if (i < n) {
                        nt = sm.pre[i + 1] - sm.pre[i];
                        enter();
                    }
                }
            }
            if (u + 1 < end) {
                tiles_of(next);
                prefetch_tile<T, D>(p.bounds, next, qd);
            }
        });
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
            size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, off));
        const int j = first + 8 * qd + r;
        if (qd < 2 && j < blocks)
            p.scores[run * p.row + j] = score_key(qd ? best[1] : best[0]);
        if (lane == 0)
            p.sizes[run * (p.row / 16) + first / 16] = size;
        tile[0] = next[0];
        tile[1] = next[1];
    }
}

template <typename T, int D, int NT, int NTH, bool SCORED>
__global__ void __launch_bounds__(NTH, SCORED ? 1 : 512 / NTH) block_select_kernel_t(const SelectParams p)
{
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int NW = NTH / 32;
    extern __shared__ uint32_t near_scores[];
    __shared__ float q[8 * NT * D];               // the group's queries
    __shared__ unsigned long long near_keys[kDoubt];
    __shared__ TallySmem<NW> counts;
    __shared__ RadixSmem<NW> radix;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv;
    Tally<NW, false> tally(counts);
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
    // the pool tile of block j; a bad entry counts as block 0
    auto tile_of = [&](int j) {
        int phys = __ldg(table + j);
        if ((unsigned)phys >= (unsigned)p.num_blocks) {
            record_error(p.err, PA_DEVERR_TABLE_RANGE);
            phys = 0;
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

    // ---- the scores ----
    uint32_t *far_scores = p.scores + (size_t)run * p.row;
    uint32_t *score = p.near >= nb ? near_scores : far_scores;
    const T *qg = static_cast<const T *>(p.q) + (size_t)run * G * D;
    float size = 0.f;                             // the largest sum |q||bound|
    uint32_t least = 0, most = 0;                 // of the finite scores, least upside down
    int infs = 0;                                 // those that are not rank first
    auto seen_score = [&](int j, uint32_t k) {
        if (k != kFirst) {
            least = max(least, ~k);
            most = max(most, k);
        } else {
            infs += j >= lo && j < hi;
        }
    };
    if (SCORED) {
        for (int i = tid; i < (nb + 15) / 16; i += NTH)
            size = fmaxf(size, __ldcg(p.sizes + (size_t)run * (p.row / 16) + i));
        const uint4 *src = reinterpret_cast<const uint4 *>(far_scores);
#pragma unroll 2
        for (int i = tid; i < (nb + 3) / 4; i += NTH) {
            const uint4 x = __ldcg(src + i);
            const uint32_t k[4] = {x.x, x.y, x.z, x.w};
            if (p.near >= nb)
                reinterpret_cast<uint4 *>(near_scores)[i] = x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * i + e < nb)
                    seen_score(4 * i + e, k[e]);
        }
    } else {
        const int r = lane >> 2, qd = lane & 3;
        ScoreQueries<T, D, NT> queries;
        queries.load(qg, G, r, qd);
        // rows r and r + 8 of the next 16 blocks; past the end the last block again
        auto rows = [&](int b, int (&tile)[2]) {
            tile[0] = tile_of(min(b + r, nb - 1));
            tile[1] = tile_of(min(b + 8 + r, nb - 1));
        };
        int tile[2] = {0, 0}, next[2] = {0, 0};
        if (16 * warp < nb)
            rows(16 * warp, tile);
        for (int b = 16 * warp; b < nb; b += 16 * NW) {
            float best[2];
            score_tile<T, D, NT>(queries, p.bounds, tile, G, qd, best, size, [&]() {
                if (b + 16 * NW < nb) {
                    rows(b + 16 * NW, next);
                    prefetch_tile<T, D>(p.bounds, next, qd);
                }
            });
            const int j = b + 8 * qd + r;
            if (qd < 2 && j < nb) {
                const uint32_t k = score_key(qd ? best[1] : best[0]);
                score[j] = k;
                seen_score(j, k);
            }
            tile[0] = next[0];
            tile[1] = next[1];
        }
    }
    // ---- the queries, for those that are summed again ----
    for (int i = tid; i < G * D; i += NTH)
        q[i] = Elem<T>::to_f(qg[i]);
    for (int i = tid; i < 2 * RadixSmem<NW>::BINS; i += NTH)
        radix.hist[0][i] = 0;
    __syncthreads();
    // a warp's contiguous part of the blocks that compete: [w0, ..) in `steps` steps of 32
    const int c1 = hi, steps = (c1 - lo + NTH - 1) / NTH;
    const int w0 = lo + warp * steps * 32;
    auto each = [&](auto &&f) {                   // f(block, score), 0 past the end
#pragma unroll 4
        for (int i = 0; i < steps; ++i) {
            const int j = w0 + 32 * i + lane;
            f(j, j < c1 ? score[j] : 0u);
        }
    };
    int all_infs, none;
    const uint3 range = tally.most(__reduce_add_sync(FULL, infs), least, most,
                                   __float_as_uint(size), all_infs, none);
    const int inf_left = min(all_infs, want);     // so many of them, the foremost
    want -= inf_left;
    int4 all, before;
    int inf_before = 0;                           // in the warps before this one
    if (all_infs > 0) {
        infs = 0;
        each([&](int, uint32_t k) { infs += k == kFirst; });
        tally.sums(__reduce_add_sync(FULL, infs), 0, 0, all, before);
        inf_before = before.x;
    }
    // Largest error: 2 D / 16 steps each add 17 terms aligned to the largest, none above
    // sum |q||bound|, and lose 2^-23 of it a term (sums that are infinite put everything in
    // doubt)
    const float twice = 2.f * (2 * D / 16) * 17 * 1.1920929e-7f * __uint_as_float(range.z);
    const float slack = twice <= FLT_MAX ? twice : FLT_MAX;
    int ins = 0, ins_before = -1;                 // kept by this warp; by those before it, if known

    // ---- a score that just `want` reach, or else the want-th largest itself ----
    uint32_t sure_above = kFirst - 1, doubt_from = kFirst - 1;   // none is kept
    if (want > 0) {
        int above, reach;
        const float edge = from_ordered(tally.threshold(
            radix,
            [&](auto &&f) { each([&](int, uint32_t k) { f(k, k != 0 && k != kFirst); }); }, want,
            ~range.x, range.y, above, reach));
        // ---- in, out, or in doubt ----
        sure_above = ordered(__fadd_ru(edge, slack));
        doubt_from = ordered(__fadd_rd(edge, -slack));
        auto doubtful = [&](uint32_t k) { return k >= doubt_from && k <= sure_above; };
        int sure = 0, doubts = 0;
        each([&](int, uint32_t k) {
            sure += k > sure_above && k != kFirst;
            doubts += doubtful(k);
        });
        sure = __reduce_add_sync(FULL, sure);
        doubts = __reduce_add_sync(FULL, doubts);
        tally.sums(sure, doubts, 0, all, before);
        const int need = want - all.x, total = all.y, mine = before.y;
        if (need == 0 || need == total) {
            // none or all of them: no sums wanted
            ins_before = before.x + (need ? before.y : 0);
            each([&](int j, uint32_t k) {
                if (need && doubtful(k))
                    score[j] = kIn;
            });
        } else {
            // the score of block j by the warp, as an ordered number of 64 bits
            auto resum = [&](int j) {
                const T *b = static_cast<const T *>(p.bounds) + (size_t)tile_of(j) * 2 * D;
                float bound[2][D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    bound[0][c] = Elem<T>::to_f(b[32 * c + lane]);
                    bound[1][c] = Elem<T>::to_f(b[D + 32 * c + lane]);
                }
                unsigned long long best = 0;
                for (int g = 0; g < G; ++g) {
                    float a = 0.f, e = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        const float qc = q[g * D + 32 * c + lane];
                        two_add(a, e, qc * (qc > 0.f ? bound[1][c] : bound[0][c]));   // exact
                    }
#pragma unroll
                    for (int off = 16; off; off >>= 1) {
                        const float oa = __shfl_xor_sync(FULL, a, off);
                        const float oe = __shfl_xor_sync(FULL, e, off);
                        two_add(a, e, oa);
                        e = __fadd_rn(e, oe);
                    }
                    const float x = __fadd_rn(a, e), rest = __fsub_rn(e, __fsub_rn(x, a));
                    const unsigned long long kk =
                        (unsigned long long)ordered(x) << 32 | ordered(rest);
                    best = kk > best ? kk : best;
                }
                // (the lanes' sums differ in their last bits: the order of their terms does)
                return __shfl_sync(FULL, best, 0);
            };
            // their keys in the order of their positions; key i of the run is in list[i]
            unsigned long long *list =
                total <= kDoubt ? near_keys : p.exact + (size_t)run * p.row;
            int at = mine;
            each([&](int j, uint32_t x) {
                unsigned m = __ballot_sync(FULL, doubtful(x));
                for (; m; m &= m - 1) {
                    const int l = __ffs(m) - 1;
                    const unsigned long long k = resum(j - lane + l);
                    if (lane == 0)
                        list[at] = k;
                    ++at;
                }
            });
            const int end = at;
            tally.sync();
            if (total <= kDoubt) {
                // rank each among all
                at = mine;
                each([&](int j, uint32_t x) {
                    unsigned m = __ballot_sync(FULL, doubtful(x));
                    uint32_t mark = x;
                    for (; m; m &= m - 1, ++at) {
                        const unsigned long long k = list[at];
                        int better = 0;
                        for (int o = lane; o < total; o += 32)
                            better += list[o] > k || (list[o] == k && o < at);
                        better = __reduce_add_sync(FULL, better);
                        if (lane == __ffs(m) - 1)
                            mark = better < need ? kIn : kOut;
                    }
                    if (mark != x)
                        score[j] = mark;
                });
            } else {
                // very many scores close together (equal blocks): the need-th largest key, two
                // bits at a time
                unsigned long long t64 = 0;
                auto count = [&](unsigned long long at_least) {
                    int n = 0;
                    for (int i = mine + lane; i < end; i += 32)
                        n += list[i] >= at_least;
                    return __reduce_add_sync(FULL, n);
                };
                for (int bit64 = 62; bit64 >= 0; bit64 -= 2) {
                    const unsigned long long t1 = t64 | 1ull << bit64, t2 = t64 | 2ull << bit64,
                                             t3 = t64 | 3ull << bit64;
                    tally.sums(count(t1), count(t2), count(t3), all, before);
                    t64 = all.z >= need ? t3 : all.y >= need ? t2 : all.x >= need ? t1 : t64;
                }
                // of those equal to it the first ones
                const int above = t64 == ~0ull ? 0 : count(t64 + 1);
                tally.sums(above, count(t64) - above, 0, all, before);
                int quota = need - all.x - before.y;
                at = mine;
                each([&](int j, uint32_t x) {
                    const bool on = doubtful(x);
                    const unsigned m = __ballot_sync(FULL, on), below = (1u << lane) - 1;
                    const unsigned long long k = on ? list[at + __popc(m & below)] : 0;
                    const unsigned tie = __ballot_sync(FULL, on && k == t64);
                    if (on)
                        score[j] = k > t64 || (k == t64 && __popc(tie & below) < quota) ? kIn : kOut;
                    quota -= __popc(tie);
                    at += __popc(m);
                });
            }
        }
        __syncwarp();                             // the marks, which the same warp reads
    }

    // ---- the kept blocks in their order ----
    int seen = inf_before;
    auto kept = [&](uint32_t k) {                 // asked in ascending order
        if (all_infs == 0)
            return k > sure_above;
        const unsigned inf = __ballot_sync(FULL, k == kFirst);
        const bool in = k == kFirst ? seen + __popc(inf & ((1u << lane) - 1)) < inf_left
                                    : k > sure_above;
        seen += __popc(inf);
        return in;
    };
    if (want == 0)
        ins_before = 0;
    if (ins_before >= 0) {
        ins_before += min(inf_before, inf_left);
    } else {
        each([&](int, uint32_t k) { ins += kept(k); });
        tally.sums(__reduce_add_sync(FULL, ins), 0, 0, all, before);
        ins_before = before.x;
    }
    int at = lo + ins_before;
    seen = inf_before;
    each([&](int j, uint32_t k) {
        const bool in = kept(k);
        const unsigned m = __ballot_sync(FULL, in);
        if (in)
            out[at + __popc(m & ((1u << lane) - 1))] = tile_of(j);
        at += __popc(m);
    });
    for (int i = tid; i < p.keep_first + p.keep_last; i += NTH)
        if (i < lo)
            out[i] = tile_of(i);
        else
            out[p.keep - p.keep_last + i - lo] = tile_of(hi + i - lo);
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

namespace {

// which: the selection with scores of its own by 128 or by 256 threads, that from given
// scores by 1024, or the kernel that computes those
enum Which { kSmall, kLarge, kGiven, kScores };

template <typename T, int D, int NT>
const void *select_fn(Which which)
{
    switch (which) {
    case kSmall:
        return reinterpret_cast<const void *>(&block_select_kernel_t<T, D, NT, 128, false>);
    case kLarge:
        return reinterpret_cast<const void *>(&block_select_kernel_t<T, D, NT, 256, false>);
    case kGiven:
        return reinterpret_cast<const void *>(&block_select_kernel_t<T, D, NT, 1024, true>);
    default:
        return reinterpret_cast<const void *>(&block_score_kernel_t<T, D, NT>);
    }
}

const void *select_fn(bool bf16, int head_dim, int group, Which which)
{
    if (head_dim == 128)
        return bf16 ? group <= 8 ? select_fn<__nv_bfloat16, 128, 1>(which)
                                 : select_fn<__nv_bfloat16, 128, 2>(which)
                    : group <= 8 ? select_fn<__half, 128, 1>(which)
                                 : select_fn<__half, 128, 2>(which);
    return bf16 ? group <= 8 ? select_fn<__nv_bfloat16, 64, 1>(which)
                             : select_fn<__nv_bfloat16, 64, 2>(which)
                : group <= 8 ? select_fn<__half, 64, 1>(which) : select_fn<__half, 64, 2>(which);
}

}  // namespace

SelectLaunch select_launch(bool bf16, int head_dim, int group, int num_runs, int max_blocks,
                           int keep, int num_sms)
{
    SelectLaunch e{};
    const bool small = max_blocks <= 256;
    // A thread block a run, or, with few runs, the scores apart: bf16, 32/8 heads x 128, lengths
    // to 16K, us in a graph of the one and of the other: 128 runs 17.4 / 14.7, 256 runs 20.2 /
    // 22.6, 512 runs 38.5 / 48.7; 32 runs of 32K to 131K tokens 98 / 24.3.  Short tables: 128
    // threads against what they would else have: 8 runs of 4096 tokens 7.8 / 8.5 (apart), 64
    // runs 10.3 / 11.9 (apart), 256 runs 12.6 / 10.6 (256 threads), 1024 runs 24.9 / 31.6, 4096
    // runs 76.6 / 104.7; 32 runs to 1024 tokens of 64 channels 4.5 / 8.6 (apart).  Long ones
    // without: 256 runs to 16K tokens 35.4 by 128 threads, 29.4 by 256; 512 runs 45.5 / 46.0.
    const bool apart = !small && max_blocks > keep && 2LL * num_runs < 3LL * num_sms &&
                       num_runs <= kRaggedSeqs;
    e.threads = small ? 128 : apart ? 1024 : 256;
    e.fn = select_fn(bf16, head_dim, group, small ? kSmall : apart ? kGiven : kLarge);
    if (apart) {
        e.score_fn = select_fn(bf16, head_dim, group, kScores);
        e.score_threads = kScoreThreads;
        // as many blocks as run at once, or as there is work for
        const long long warps = (long long)num_runs * ((max_blocks + 15) / 16);
        const long long blocks = (warps + kScoreThreads / 32 - 1) / (kScoreThreads / 32);
        e.score_blocks = (int)(blocks < 4LL * num_sms ? blocks : 4LL * num_sms);
    }
    const long long all = ((long long)max_blocks + 15) / 16 * 16;
    e.near = all <= kSelectNear ? (int)all : 0;
    e.smem = 4 * (size_t)e.near;
    return e;
}

}  // namespace pa
