// pa_tally.cuh -- counting over the warps of a thread block, or of a cluster
// of blocks, that share out one list in order: the block `rank` of the cluster
// and the warp of the block say who comes before whom.
#pragma once

#include "pa_device.cuh"

namespace pa {

template <int NW>
struct TallySmem {
    int part[2][3][NW];
    int4 total[2];                 // read by the other blocks of the cluster
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

    // The largest of three unsigned values over all warps.
    __device__ __forceinline__ uint3 most(uint32_t a, uint32_t b, uint32_t d)
    {
        constexpr uint32_t FULL = 0xffffffffu;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int(*c)[NW] = sm.part[round & 1];
        a = __reduce_max_sync(FULL, a);
        b = __reduce_max_sync(FULL, b);
        d = __reduce_max_sync(FULL, d);
        if (lane == 0) {
            c[0][warp] = (int)a;
            c[1][warp] = (int)b;
            c[2][warp] = (int)d;
        }
        __syncthreads();
        auto over = [&](int row) {
            return __reduce_max_sync(FULL, lane < NW ? (uint32_t)c[row][lane] : 0u);
        };
        uint3 all = make_uint3(over(0), over(1), over(2));
        if (CLUSTER) {
            if (threadIdx.x == 0)
                sm.total[round & 1] = make_int4((int)all.x, (int)all.y, (int)all.z, 0);
            cluster_arrive();
            cluster_wait();
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < blocks)
                y = cluster_load4(cluster_addr(smem_addr(&sm.total[round & 1]), lane));
            all = make_uint3(__reduce_max_sync(FULL, __float_as_uint(y.x)),
                             __reduce_max_sync(FULL, __float_as_uint(y.y)),
                             __reduce_max_sync(FULL, __float_as_uint(y.z)));
        }
        ++round;
        return all;
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
