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
#include <float.h>

#include "pa_device.cuh"
#include "pa_sparse.h"

namespace pa {

namespace {

constexpr int kEvictThreads = 1024;

// The order of masses as unsigned numbers: -0 as 0, a NaN above all.
__device__ __forceinline__ uint32_t mass_key(float x)
{
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return x != x ? 0xffffffffu : u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int D>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel_t(const EvictParams p)
{
    constexpr int NTH = kEvictThreads, NW = NTH / 32;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int KR = 8;                         // keys a thread holds in registers
    constexpr int CPR = D / 8;                    // 16-byte chunks of a row
    constexpr int RPW = 32 / (2 * CPR);           // tokens (K and V row) a warp moves at once
    constexpr int U = 8;                          // loads in flight a lane
    static_assert(NW == 32, "a lane reads each warp's count");
    __shared__ int part[2][3][NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.num_kv_heads;
    const int run = blockIdx.x, s = run / Hkv, h = run % Hkv;
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
    // a table that does not hold leaves the sequence as it was
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks;
    bool bad = false;
    for (int j = tid; j < (L + kBlockSize - 1) / kBlockSize; j += NTH)
        bad |= (unsigned)__ldg(table + j) >= (unsigned)p.num_blocks;
    if (__syncthreads_or(bad)) {
        if (tid == 0)
            record_error(p.err, PA_DEVERR_TABLE_RANGE);
        return;
    }
    const int R = min(p.keep_last, B), F = min(p.keep_first, B - R);
    const int edge = B - R, want = edge - F, hi = L - R;   // slots [F, hi) compete for `want`
    float *mass = p.mass + (size_t)run * p.max_blocks * kBlockSize;

    // this thread's slots: F + seg * warp + 32 i + lane, i < steps
    const int steps = ((hi - F + NW - 1) / NW + 31) / 32;
    const int slot0 = F + warp * steps * 32 + lane;
    uint32_t reg[KR];
#pragma unroll
    for (int i = 0; i < KR; ++i)
        reg[i] = i < steps && slot0 + 32 * i < hi ? mass_key(__ldcg(mass + slot0 + 32 * i)) : 0;
    auto each = [&](auto &&f) {                   // f(slot, key) over this thread's slots
#pragma unroll
        for (int i = 0; i < KR; ++i)
            if (i < steps)
                f(slot0 + 32 * i, reg[i]);
        for (int i = KR; i < steps; ++i) {
            const int t = slot0 + 32 * i;
            f(t, t < hi ? mass_key(__ldcg(mass + t)) : 0u);
        }
    };

    // the want-th largest key, two bits at a time: how many keys reach each of three
    // thresholds.  (A slot past hi has key 0, which no threshold lets through.)
    uint32_t T = 0;
    int above = 0;                                // keys >= T + 1 at the end
    if (want > 0) {
        for (int bit = 30, round = 0; bit >= 0; bit -= 2, ++round) {
            const uint32_t t1 = T | 1u << bit, t2 = T | 2u << bit, t3 = T | 3u << bit;
            int n1 = 0, n2 = 0, n3 = 0;
            each([&](int, uint32_t k) {
                n1 += k >= t1;
                n2 += k >= t2;
                n3 += k >= t3;
            });
            n1 = __reduce_add_sync(FULL, n1);
            n2 = __reduce_add_sync(FULL, n2);
            n3 = __reduce_add_sync(FULL, n3);
            int(*c)[NW] = part[round & 1];
            if (lane == 0) {
                c[0][warp] = n1;
                c[1][warp] = n2;
                c[2][warp] = n3;
            }
            __syncthreads();
            n1 = __reduce_add_sync(FULL, c[0][lane]);
            n2 = __reduce_add_sync(FULL, c[1][lane]);
            n3 = __reduce_add_sync(FULL, c[2][lane]);
            // (a NaN's key is all ones: T + 1 is never asked for it)
            T = n3 >= want ? t3 : n2 >= want ? t2 : n1 >= want ? t1 : T;
        }
        int n = 0;
        each([&](int, uint32_t k) { n += k > T; });
        n = __reduce_add_sync(FULL, n);
        if (lane == 0)
            part[0][0][warp] = n;
        __syncthreads();
        above = __reduce_add_sync(FULL, part[0][0][lane]);
        __syncthreads();
    }
    // of the keys equal to T the first ones: this warp's share of them
    auto before_me = [&](int mine, int buf, int row) {
        if (lane == 0)
            part[buf][row][warp] = mine;
        __syncthreads();
        return __reduce_add_sync(FULL, lane < warp ? part[buf][row][lane] : 0);
    };
    int ties = 0;
    each([&](int t, uint32_t k) { ties += __popc(__ballot_sync(FULL, t < hi && k == T)); });
    int quota = want - above - before_me(ties, 1, 0);
    quota = want > 0 ? max(0, quota) : 0;
    // kept(slot, key), to be asked in ascending order of the slots
    int used = 0;
    auto kept = [&](int t, uint32_t k) {
        const unsigned tie = __ballot_sync(FULL, want > 0 && t < hi && k == T);
        const bool in = want > 0 && t < hi &&
                        (k > T || (k == T && used + __popc(tie & ((1u << lane) - 1)) < quota));
        used += __popc(tie);
        return in;
    };
    int holes = 0, movers = 0;
    each([&](int t, uint32_t k) {
        const bool in = kept(t, k);
        holes += __popc(__ballot_sync(FULL, !in && t < edge));
        movers += __popc(__ballot_sync(FULL, in && t >= edge));
    });
    int hole = before_me(holes, 1, 1), mover = before_me(movers, 1, 2);
    const int moves = __reduce_add_sync(FULL, part[1][2][lane]);
    int32_t *to = p.lists + (size_t)run * 2 * p.list, *from = to + p.list;
    used = 0;
    each([&](int t, uint32_t k) {
        const bool in = kept(t, k);
        const unsigned below = (1u << lane) - 1;
        const unsigned hb = __ballot_sync(FULL, !in && t < edge);
        const unsigned mb = __ballot_sync(FULL, in && t >= edge);
        if (!in && t < edge)
            to[hole + __popc(hb & below)] = t;
        if (in && t >= edge)
            from[mover + __popc(mb & below)] = t;
        hole += __popc(hb);
        mover += __popc(mb);
    });
    __syncthreads();

    // a lane's 16 bytes of a token's K row or V row
    const int sub = lane / (2 * CPR), ch = lane % (2 * CPR);
    uint4 *pool = static_cast<uint4 *>(ch < CPR ? p.k_cache : p.v_cache) + ch % CPR;
    auto row_of = [&](int t) {
        return pool + (((size_t)__ldg(table + t / kBlockSize) * Hkv + h) * kBlockSize +
                       t % kBlockSize) * CPR;
    };
    for (int base = warp * RPW + sub; base < moves; base += NW * RPW * U) {
        uint4 x[U];
        float m[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = base + i * NW * RPW;
            if (j < moves) {
                const int t = __ldcg(from + j);
                x[i] = __ldcg(row_of(t));
                if (ch == 0)
                    m[i] = __ldcg(mass + t);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = base + i * NW * RPW;
            if (j < moves) {
                const int t = __ldcg(to + j);
                *row_of(t) = x[i];
                if (ch == 0)
                    mass[t] = m[i];
            }
        }
    }
    // The last ones move down by L - B.  Rounds in ascending order, each loaded whole before
    // it is stored: a round's destinations lie before every later round's sources.
    __syncthreads();
    for (int base = 0; base < R; base += NW * RPW * U) {
        uint4 x[U];
        float m[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = base + (i * NW + warp) * RPW + sub;
            if (j < R) {
                x[i] = __ldcg(row_of(hi + j));
                if (ch == 0)
                    m[i] = __ldcg(mass + hi + j);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = base + (i * NW + warp) * RPW + sub;
            if (j < R) {
                *row_of(edge + j) = x[i];
                if (ch == 0)
                    mass[edge + j] = m[i];
            }
        }
    }
}

}  // namespace

SparseKernel evict_kernel(int head_dim)
{
    return SparseKernel{head_dim == 128
                            ? reinterpret_cast<const void *>(&evict_kernel_t<128>)
                            : reinterpret_cast<const void *>(&evict_kernel_t<64>),
                        kEvictThreads};
}

}  // namespace pa
