// pa_evict.cu -- a sequence of the paged pool shortened in place to the tokens
// with the largest accumulated attention weight (sm_103a).
//
// Of L tokens B stay: the keep_first first ones, the keep_last last ones and of
// the rest those with the largest mass.  Attention does not ask for the order of the
// keys (their positions are in their rotation), so as little moves as can: the
// last ones, in their order, to the new end, and what is kept from beyond the
// new end into the holes that dropped tokens left before it.  The sources of those
// moves lie past all of their destinations, so they need no order among
// themselves.
#include <limits.h>

#include "pa_device.cuh"
#include "pa_sparse.h"
#include "pa_tally.cuh"

namespace pa {

namespace {

// Holes and sources up to this many a run stay in shared memory, others in the workspace.
constexpr int kEvictList = 256;

// The order of masses as unsigned numbers: -0 as 0, a NaN above all.
__device__ __forceinline__ uint32_t mass_key(float x)
{
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return x != x ? 0xffffffffu : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One (sequence, kv head) per thread block, or per cluster of blocks that share out its
// slots and its moves (CLUSTER).  The choice is a chain of passes over the keys in shared
// memory, a barrier each (two to four digits of a histogram, ties, holes and movers); the moves
// are bound by HBM where many rows move (128 x 4096 tokens to 2048: 1.15 GB read and written in
// 197 us, 5.8 TB/s).  A batch of 128 that gives back one block, 47 rows a run, 55 MB, 17.3 us: half
// the choice.  (Here and below: K, V and masses renewed before each call and none of them in
// L2; a second call on the same masses finds most of the heavy tokens moved.)
template <int D, int NTH, bool CLUSTER>
__global__ void __launch_bounds__(NTH) evict_kernel_t(const EvictParams p)
{
    constexpr int NW = NTH / 32;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int CPR = D / 8;                    // 16-byte chunks of a row
    constexpr int RPW = 32 / (2 * CPR);           // tokens (K and V row) a warp loads at once
    constexpr int U = 8;                          // loads in flight a lane
    // keys of the block's slots (p.keys of them), the table, holes and sources
    extern __shared__ uint32_t smem[];
    uint32_t *keys = smem;
    int32_t *sm_table = reinterpret_cast<int32_t *>(smem + p.keys);
    int32_t *sm_list = sm_table + p.table;
    __shared__ TallySmem<NW> counts;
    __shared__ RadixSmem<NW> radix;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.num_kv_heads;
    Tally<NW, CLUSTER> tally(counts);
    const int C = tally.blocks, rank = tally.rank;
    const int run = blockIdx.x / C, s = run / Hkv, h = run % Hkv;
    grid_dependents_launch();
    grid_dependency_wait();
    const int L = __ldg(p.seq_lens + s);
    const int B = __ldg(p.new_lens + s);
    if (L < 0 || L > p.max_blocks * kBlockSize || B < 0) {
        if (tid == 0)
            record_error(p.err, PA_DEVERR_SEQLEN_RANGE);
        return;
    }
    if (B >= L)
        return;
    const int R = min(p.keep_last, B), F = min(p.keep_first, B - R);
    const int edge = B - R, want = edge - F, hi = L - R;   // slots [F, hi) compete for `want`
    float *mass = p.mass + (size_t)run * p.max_blocks * kBlockSize;

    // the block's slots [lo, end), in it a warp's [w0, w1): steps of 32, the first p.keys of
    // the block's keys in shared memory
    const int span = ((hi - F + C * NTH - 1) / (C * NTH)) * NTH;
    const int lo = min(hi, F + rank * span), end = min(hi, lo + span);
    const int steps = span / NTH;
    const int w0 = lo + warp * steps * 32;
    // a table that does not hold leaves the sequence as it was
    const int32_t *gtable = p.block_tables + (size_t)s * p.max_blocks;
    const bool near = p.table > 0;
    bool bad = false;
    constexpr int K = 8;                          // loads in flight a thread
    for (int j0 = tid; j0 < (L + kBlockSize - 1) / kBlockSize; j0 += K * NTH) {
        int b[K];
#pragma unroll
        for (int i = 0; i < K; ++i)
            b[i] = j0 + i * NTH < (L + kBlockSize - 1) / kBlockSize ? __ldg(gtable + j0 + i * NTH) : 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            bad |= (unsigned)b[i] >= (unsigned)p.num_blocks;
            if (near && j0 + i * NTH < p.table)
                sm_table[j0 + i * NTH] = b[i];
        }
    }
    const int kept_keys = min(end - lo, p.keys);
    uint32_t least = 0, most = 0;                 // of this thread's keys, least upside down
    for (int t0 = tid; t0 < kept_keys; t0 += K * NTH) {
        float m[K];
#pragma unroll
        for (int i = 0; i < K; ++i)
            m[i] = t0 + i * NTH < kept_keys ? __ldcg(mass + lo + t0 + i * NTH) : 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (t0 + i * NTH < kept_keys) {
                const uint32_t k = mass_key(m[i]);
                keys[t0 + i * NTH] = k;
                least = max(least, ~k);
                most = max(most, k);
            }
    }
    const bool all_near = end - lo <= p.keys;
    for (int t = lo + kept_keys + tid; t < end; t += NTH) {
        const uint32_t k = mass_key(__ldcg(mass + t));
        least = max(least, ~k);
        most = max(most, k);
    }
    for (int i = tid; i < 2 * RadixSmem<NW>::BINS; i += NTH)
        radix.hist[0][i] = 0;
    if (__syncthreads_or(bad)) {                  // (the same in every block of the cluster)
        if (tid == 0)
            record_error(p.err, PA_DEVERR_TABLE_RANGE);
        return;
    }
    const int32_t *table = near ? sm_table : gtable;
    auto key_of = [&](int t) {                    // past the end 0, below every real key
        return t >= end ? 0u : t - lo < p.keys ? keys[t - lo] : mass_key(__ldcg(mass + t));
    };
    auto each = [&](auto &&f) {                   // f(slot, key) over the warp's slots
        if (all_near) {
            const uint32_t *k = keys + (w0 - lo) + lane;
#pragma unroll 4
            for (int i = 0; i < steps; ++i) {
                const int t = w0 + 32 * i + lane;
                f(t, t < end ? k[32 * i] : 0u);
            }
        } else {
            for (int i = 0; i < steps; ++i) {
                const int t = w0 + 32 * i + lane;
                f(t, key_of(t));
            }
        }
    };
    // the want-th largest key: what is above it is kept, and of those equal to it the first
    // ones (just all, if no more than `want` reach it)
    uint32_t T = 0xffffffffu;
    int4 all, before;
    int quota = 0;
    if (want > 0) {
        int above, reach, none;
        const uint3 range = tally.most(0, least, most, 0u, none, none);
        T = tally.threshold(
            radix, [&](auto &&f) { each([&](int t, uint32_t k) { f(k, t < end); }); }, want,
            ~range.x, range.y, above, reach);
        quota = INT_MAX;
        if (reach != want) {
            int ties = 0;
            each([&](int t, uint32_t k) { ties += t < end && k == T; });
            tally.sums(__reduce_add_sync(FULL, ties), 0, 0, all, before);
            quota = max(0, want - above - before.x);
        }
    }
    int used = 0;
    auto kept = [&](int t, uint32_t k) {          // asked in ascending order
        bool tied = t < end && k == T;
        if (quota != INT_MAX) {
            const unsigned tie = __ballot_sync(FULL, tied);
            tied = tied && used + __popc(tie & ((1u << lane) - 1)) < quota;
            used += __popc(tie);
        }
        return t < end && (k > T || tied);
    };
    int holes = 0, movers = 0;
    each([&](int t, uint32_t k) {
        const bool in = kept(t, k);
        holes += !in && t < min(edge, end);
        movers += in && t >= edge;
    });
    tally.sums(__reduce_add_sync(FULL, holes), __reduce_add_sync(FULL, movers), 0, all, before);
    const int moves = all.y;
    int hole = before.x, mover = before.y;
    const bool few = !CLUSTER && moves <= kEvictList;
    int32_t *to = few ? sm_list : p.lists + (size_t)run * 2 * p.list;
    int32_t *from = to + (few ? kEvictList : p.list);
    used = 0;
    if (moves > 0)
        each([&](int t, uint32_t k) {
            const bool in = kept(t, k), is_hole = !in && t < min(edge, end), moving = in && t >= edge;
            const unsigned below = (1u << lane) - 1;
            const unsigned hb = __ballot_sync(FULL, is_hole), mb = __ballot_sync(FULL, moving);
            if (is_hole)
                to[hole + __popc(hb & below)] = t;
            if (moving)
                from[mover + __popc(mb & below)] = t;
            hole += __popc(hb);
            mover += __popc(mb);
        });
    tally.sync();

    // The moves, then the last ones' way down by L - B, in rounds that are loaded whole before
    // they are stored: what a round writes lies before all that later rounds read.  A warp takes
    // neighbouring moves, a lane holds one's places (the next round's are fetched ahead) and its
    // mass, and takes 16 bytes of a token's K row or V row.
    constexpr int WT = U * RPW;                   // tokens of a warp's round
    const int sub = lane / (2 * CPR), ch = lane % (2 * CPR);
    uint4 *pool = static_cast<uint4 *>(ch < CPR ? p.k_cache : p.v_cache) + ch % CPR;
    auto row_of = [&](int t) {
        return pool + (((size_t)table[t / kBlockSize] * Hkv + h) * kBlockSize + t % kBlockSize) * CPR;
    };
    const int per = C * NW * WT;                  // tokens the run's warps take at once
    auto places = [&](int base, int &src, int &dst) {
        const int j = base + (rank * NW + warp) * WT + lane;
        src = dst = -1;
        if (lane < WT && j < moves + R) {
            src = j < moves ? from[j] : hi + j - moves;
            dst = j < moves ? to[j] : edge + j - moves;
        }
    };
    int src, dst, src_next, dst_next;
    places(0, src, dst);
    for (int base = 0; base < moves + R; base += per) {
        uint4 x[U];
        const float m = dst >= 0 ? __ldcg(mass + src) : 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int at = __shfl_sync(FULL, src, i * RPW + sub);
            if (at >= 0)
                x[i] = __ldcg(row_of(at));
        }
        places(base + per, src_next, dst_next);
        if (base + per > moves)                   // the last ones: their places may be read here
            tally.sync();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int at = __shfl_sync(FULL, dst, i * RPW + sub);
            if (at >= 0)
                *row_of(at) = x[i];
        }
        if (dst >= 0)
            mass[dst] = m;
        src = src_next;
        dst = dst_next;
    }
    tally.leave();
}

constexpr int kEvictKeys = 32768;                 // keys a block holds (128 KB)
constexpr int kEvictTable = 8192;                 // table entries a block holds (32 KB)

}  // namespace

// 256 threads a block, four of which an SM holds; where the runs leave SMs idle, or a run's
// masses would take much of an SM's shared memory, a cluster of 2, 4 or 8 blocks shares one.
// More than three short runs an SM: 128 threads, eight blocks an SM.  us in a graph, bf16, 8 heads x
// 128, sequences x tokens -> kept.  128 / 256 threads: 128 x 1040 -> 1024 17.3 / 22.0, 128 x 2048
// -> 2030 27.5 / 32.0, 128 x 2048 -> 1024 113 / 107, 32 x 1040 -> 1024 12.7 / 12.5, 4 x 2000 -> 1024
// 33.8 / 19.7.  1 / 2 / 4 / 8 blocks: 4 x 4096 -> 2048 34.0 / 24.2 / 22.2 / 20.9, 32 x 2048 -> 2030
// 14.2 / 14.8 / 24.6 / 46.5, 16 x 8192 -> 8000 24.8 / 23.0 / 19.6 / 31.9, 8 x 32K -> 2048 96.2 /
// 62.4 / 53.0 / 41.7, 32 x 32K -> 4096 297 / 220 / 224 / 210, 128 x 16K -> 2048 421 / 367 / 370 /
// 413, 64 x 8192 -> 2048 158 / 162 / 170 / 198, 128 x 4096 -> 2048 200 / 209 / 227 / 303.
EvictLaunch evict_launch(int head_dim, int num_runs, int max_blocks, int num_sms)
{
    EvictLaunch e{};
    const long long slots = (long long)max_blocks * kBlockSize;
    const bool small = slots <= 2048 && num_runs > 3LL * num_sms;
    e.threads = small ? 128 : 256;
    e.cluster = 1;
    while (!small && e.cluster < 8 &&
           ((2LL * e.cluster * num_runs <= 4LL * num_sms && slots >= 4096LL * e.cluster) ||
            (2LL * e.cluster * num_runs <= num_sms && slots >= 2048LL * e.cluster) ||
            slots >= 16384LL * e.cluster))
        e.cluster *= 2;
    if (small)
        e.fn = head_dim == 128 ? reinterpret_cast<const void *>(&evict_kernel_t<128, 128, false>)
                               : reinterpret_cast<const void *>(&evict_kernel_t<64, 128, false>);
    else
        e.fn = head_dim == 128 ? reinterpret_cast<const void *>(&evict_kernel_t<128, 256, true>)
                               : reinterpret_cast<const void *>(&evict_kernel_t<64, 256, true>);
    const long long share = (slots + (long long)e.cluster * e.threads - 1) /
                            ((long long)e.cluster * e.threads) * e.threads;
    e.keys = (int)(share < kEvictKeys ? share : kEvictKeys);
    e.table = max_blocks <= kEvictTable ? max_blocks : 0;
    e.smem = 4 * ((size_t)e.keys + e.table + 2 * kEvictList);
    return e;
}

}  // namespace pa
