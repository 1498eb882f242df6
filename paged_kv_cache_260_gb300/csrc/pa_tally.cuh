// pa_tally.cuh -- counting over the warps of a thread block, or of a cluster
// of blocks, that share out one list in order: the block `rank` of the cluster
// and the warp of the block say who comes before whom.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kTallyBlocks = 8;    // most blocks of a cluster

template <int NW>
struct TallySmem {
    int part[2][4][NW];
    int4 total[2];                 // read by the other blocks of the cluster
};

// How many keys have each value of a digit, a thread's values one after the other; 32
// values a group.
template <int NW>
struct RadixSmem {
    static constexpr int BITS = NW == 4 ? 9 : 10, BINS = 1 << BITS, GROUPS = BINS / 32;
    static constexpr int EACH = BINS / (32 * NW);          // values a thread
    static_assert(NW == 4 || NW == 8 || NW == 16 || NW == 32, "128 to 1024 threads");
    int hist[2][BINS];
    int group[2][GROUPS];          // both read by the other blocks of the cluster
    int found[3];
};

template <int NW, bool CLUSTER>
struct Tally {
    TallySmem<NW> &sm;
    int blocks, rank;              // of the cluster; 1 and 0 without one
    int round = 0;                 // picks one of two buffers: one barrier a call

    __device__ __forceinline__ explicit Tally(TallySmem<NW> &s)
        : sm(s), blocks(CLUSTER ? (int)cluster_size() : 1),
          rank(CLUSTER ? (int)cluster_rank() : 0)
    {
    }

    // Three warp-uniform counts of every warp: their sums over all warps, and over those
    // before this one.  Called by every thread; what threads wrote to shared memory, and in a
    // cluster to global memory, before the call is seen after it.
    __device__ __forceinline__ void sums(int n1, int n2, int n3, int4 &all, int4 &before)
    {
        constexpr uint32_t FULL = 0xffffffffu;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int(*c)[NW] = sm.part[round & 1];
        if (lane == 0) {
            c[0][warp] = n1;
            c[1][warp] = n2;
            c[2][warp] = n3;
        }
        __syncthreads();
        auto over = [&](int row, int below) {
            return __reduce_add_sync(FULL, lane < below ? c[row][lane] : 0);
        };
        all = make_int4(over(0, NW), over(1, NW), over(2, NW), 0);
        before = make_int4(over(0, warp), over(1, warp), over(2, warp), 0);
        if (CLUSTER) {
            if (threadIdx.x == 0)
                sm.total[round & 1] = all;
            cluster_arrive();
            cluster_wait();
            int4 x = make_int4(0, 0, 0, 0);
            if (lane < blocks) {
                const float4 y = cluster_load4(cluster_addr(smem_addr(&sm.total[round & 1]), lane));
                x = make_int4(__float_as_int(y.x), __float_as_int(y.y), __float_as_int(y.z), 0);
            }
            auto add = [&](int v, bool on) { return __reduce_add_sync(FULL, on ? v : 0); };
            all = make_int4(add(x.x, true), add(x.y, true), add(x.z, true), 0);
            before.x += add(x.x, lane < rank);
            before.y += add(x.y, lane < rank);
            before.z += add(x.z, lane < rank);
        }
        ++round;
    }

    // A count's sum over all warps and over those before this one, and the largest of three
    // unsigned values.
    __device__ __forceinline__ uint3 most(int n, uint32_t a, uint32_t b, uint32_t d, int &all,
                                          int &before)
    {
        constexpr uint32_t FULL = 0xffffffffu;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int(*c)[NW] = sm.part[round & 1];
        a = __reduce_max_sync(FULL, a);
        b = __reduce_max_sync(FULL, b);
        d = __reduce_max_sync(FULL, d);
        if (lane == 0) {
            c[0][warp] = n;
            c[1][warp] = (int)a;
            c[2][warp] = (int)b;
            c[3][warp] = (int)d;
        }
        __syncthreads();
        auto over = [&](int row) {
            return __reduce_max_sync(FULL, lane < NW ? (uint32_t)c[row][lane] : 0u);
        };
        uint3 top = make_uint3(over(1), over(2), over(3));
        all = __reduce_add_sync(FULL, lane < NW ? c[0][lane] : 0);
        before = __reduce_add_sync(FULL, lane < warp ? c[0][lane] : 0);
        if (CLUSTER) {
            if (threadIdx.x == 0)
                sm.total[round & 1] = make_int4(all, (int)top.x, (int)top.y, (int)top.z);
            cluster_arrive();
            cluster_wait();
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < blocks)
                y = cluster_load4(cluster_addr(smem_addr(&sm.total[round & 1]), lane));
            all = __reduce_add_sync(FULL, __float_as_int(y.x));
            before += __reduce_add_sync(FULL, lane < rank ? __float_as_int(y.x) : 0);
            top = make_uint3(__reduce_max_sync(FULL, __float_as_uint(y.y)),
                             __reduce_max_sync(FULL, __float_as_uint(y.z)),
                             __reduce_max_sync(FULL, __float_as_uint(y.w)));
        }
        ++round;
        return top;
    }

    // A threshold that just `want` keys reach, or else the want-th largest key itself: digit
    // by digit from the top, each round counts the keys of every value of the next digit, among
    // those that share the digits found so far.  least and most are the smallest and the
    // largest key; the digits are those of key - least, so that the first one already
    // spreads the keys over its values (the leading bits of floats of one size are the
    // same, and a count that all threads add to one at a time takes its time).  There are
    // `want` > 0 keys at least.  each(f) calls f(key, whether it counts) for the caller's
    // keys.  r.hist is zero and seen to be.  above: keys larger than the threshold's digits;
    // reach: keys that are not smaller, -1 if all keys are equal.
    template <typename F>
    __device__ __forceinline__ uint32_t threshold(RadixSmem<NW> &r, const F &each, int want,
                                                  uint32_t least, uint32_t most, int &above,
                                                  int &reach)
    {
        constexpr uint32_t FULL = 0xffffffffu;
        constexpr int BITS = RadixSmem<NW>::BITS;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        above = 0;
        reach = -1;
        uint32_t t = 0;
        int bits = 32 - __clz(most - least);
        for (int buf = 0; bits > 0 && reach != want; buf ^= 1) {
            const int shift = max(0, bits - BITS);
            const uint32_t mask = (1u << (bits - shift)) - 1u;
            int *hist = r.hist[buf];
            const uint32_t high = bits < 32 ? t >> bits : 0u;
            each([&](uint32_t k, bool on) {
                k -= least;
                if (on && (bits < 32 ? k >> bits : 0u) == high)
                    atomicAdd(&hist[k >> shift & mask], 1);
            });
            __syncthreads();
            constexpr int EACH = RadixSmem<NW>::EACH, SPAN = 32 / EACH;
            int n = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                n += hist[EACH * threadIdx.x + i];
#pragma unroll
            for (int o = 1; o < SPAN; o <<= 1)
                n += __shfl_xor_sync(FULL, n, o);
            if (lane % SPAN == 0)
                r.group[buf][threadIdx.x / SPAN] = n;
            sync();
            // (the blocks have read the other buffer: they have been through this barrier)
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                r.hist[buf ^ 1][EACH * threadIdx.x + i] = 0;
            if (warp == 0) {
                // the group with the want-th largest, then the value: a lane each, summed over
                // the blocks with all loads in flight at once
                int value = 0, over = above, top = 0;
#pragma unroll
                for (int level = 0; level < 2; ++level) {
                    const int *row = level ? hist + 32 * value : r.group[buf];
                    const bool on = level || lane < RadixSmem<NW>::GROUPS;
                    int count = 0;
                    if (CLUSTER) {
                        int y[kTallyBlocks];
#pragma unroll
                        for (int c = 0; c < kTallyBlocks; ++c)
                            y[c] = c < blocks && on ? __float_as_int(cluster_load(
                                                          cluster_addr(smem_addr(row + lane), c)))
                                                    : 0;
#pragma unroll
                        for (int c = 0; c < kTallyBlocks; ++c)
                            count += y[c];
                    } else if (on) {
                        count = row[lane];
                    }
                    int incl = count;             // of this value and those above it
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_down_sync(FULL, incl, o);
                        if (lane + o < 32)
                            incl += y;
                    }
                    // the highest lane that, with all above it, has enough
                    const int at = 31 - __clz(__ballot_sync(FULL, over + incl >= want));
                    top = over + __shfl_sync(FULL, incl, at);
                    over = top - __shfl_sync(FULL, count, at);
                    value = 32 * value + at;
                }
                if (lane == 0) {
                    r.found[0] = value;
                    r.found[1] = over;
                    r.found[2] = top;
                }
            }
            __syncthreads();
            t |= (uint32_t)r.found[0] << shift;
            above = r.found[1];
            reach = r.found[2];
            bits = shift;
        }
        return t + least;
    }

    // A barrier of the block, or of the cluster.
    __device__ __forceinline__ void sync()
    {
        if (CLUSTER) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    }

    // No block leaves while another reads its counts.
    __device__ __forceinline__ void leave()
    {
        if (CLUSTER)
            sync();
    }
};

}  // namespace pa
