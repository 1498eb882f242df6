// pa_rope.cu -- new tokens' queries and keys normalised and rotated in one
// pass, and, with slots, the keys and values written into the block pool
// (pa_rope_and_cache, pa_qk_norm_rope).
//
// The mathematics, per token at position m and per segment x of d channels (a
// head, or each of its num_maps equal parts), in fp32 with one rounding at
// the end:
//     y_c  = x_c w_c / sqrt(mean_c x_c^2 + eps)          (with a norm weight)
//     y'_a = y_a cos(m f_i) - y_b sin(m f_i)
//     y'_b = y_b cos(m f_i) + y_a sin(m f_i)             pair i < rotary_dim / 2
// The pair is (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved;
// channels past rotary_dim are only normalised.  cos and sin come from the
// caller's fp32 table, so far positions lose nothing to an angle reduced in
// 32 bits.
//
// Every element is read once and written once, and there are a handful of
// operations per element, so HBM bounds the kernel (and for a decode step's
// few tokens, the launch).
#include "pa_device.cuh"
#include "pa_rope.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;

// eight 16-bit channels to fp32 and back
template <typename T>
__device__ __forceinline__ void widen8(const uint4 &v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Elem<T>::to_f2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 narrow8(const float *x)
{
    return make_uint4(Mma<T>::pack(x[0], x[1]), Mma<T>::pack(x[2], x[3]),
                      Mma<T>::pack(x[4], x[5]), Mma<T>::pack(x[6], x[7]));
}

// One warp takes a unit: U x (32 / TS) consecutive segments of one token's
// [q | k | v] list, TS = d / 16 lanes a segment.  A lane owns two 16-byte
// vectors of its segment, placed so that it holds both channels of every pair
// it rotates: vectors (t, t + rotary_dim / 16) half-split, any two when
// interleaved.  So a rotation needs no data from another lane, and a lane reads
// and writes the same elements only (q_out may be q).
template <typename T, int TS, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel_t(const RopeParams p)
{
    constexpr int GPW = 32 / TS;              // segments a warp handles at a time
    constexpr int d = 16 * TS;
    constexpr uint32_t FULL = 0xffffffffu;
    grid_dependents_launch();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, t = lane % TS, grp = lane / TS;
    const int segs = p.q_segs + p.k_segs + p.v_segs;
    const unsigned chunks = (unsigned)(segs + U * GPW - 1) / (U * GPW);
    const unsigned units = chunks * (unsigned)p.num_tokens;
    const unsigned warps = gridDim.x * (kRopeThreads / 32);
    const int rot16 = p.rotary_dim / 16;
    // this lane's vectors of a q or k segment (v: t and t + TS)
    int va, vb;
    if constexpr (INTER) {
        va = t;
        vb = t + TS;
    } else {
        // lanes past the rotated channels take the vectors left over, two each
        va = t < rot16 ? t : 2 * t;
        vb = t < rot16 ? t + rot16 : 2 * t + 1;
    }
    for (unsigned unit = blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32; unit < units;
         unit += warps) {
        const unsigned tok = unit / chunks;
        const int seg0 = (int)(unit - tok * chunks) * (U * GPW) + grp;
        const int pos = __ldg(p.positions + tok);
        const int64_t slot = p.slots ? __ldg(p.slots + tok) : 0;
        bool live = pos >= 0 && slot >= 0;    // else a padding token: nothing read or written
        if (live && pos >= p.max_position) {
            live = false;
            if (seg0 == 0 && t == 0)
                record_error(p.err, PA_DEVERR_POSITION_RANGE);
        }
        if (live && p.slots && slot >= p.num_slots) {
            live = false;
            if (seg0 == 0 && t == 0)
                record_error(p.err, PA_DEVERR_SLOT_RANGE);
        }
        if (!live)
            continue;                         // the same for the whole warp
        uint4 xa[U], xb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int seg = seg0 + u * GPW;
            if (seg >= segs)
                continue;
            const T *row;
            int a = va, b = vb;
            if (seg < p.q_segs) {
                row = static_cast<const T *>(p.q) + tok * p.q_stride + seg * d;
            } else if (seg < p.q_segs + p.k_segs) {
                row = static_cast<const T *>(p.k) + tok * p.k_stride + (seg - p.q_segs) * d;
            } else {
                row = static_cast<const T *>(p.v) + tok * p.v_stride +
                      (seg - p.q_segs - p.k_segs) * d;
                a = t;
                b = t + TS;
            }
            xa[u] = reinterpret_cast<const uint4 *>(row)[a];
            xb[u] = reinterpret_cast<const uint4 *>(row)[b];
        }
        // the lane's eight pairs' cosines and sines, the same for every head
        float c[8], s[8];
        const float *cs = p.cos_sin + (long long)pos * p.rotary_dim;
        // first pair of each vector: half-split pairs 8t .. 8t + 7 lie across both
        const int pa0 = INTER ? 4 * va : 8 * t, pb0 = INTER ? 4 * vb : 8 * t + 4;
        const bool ra = INTER ? va < 2 * rot16 : t < rot16;
        const bool rb = INTER ? vb < 2 * rot16 : t < rot16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        if (ra) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(cs + pa0));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(cs + p.rotary_dim / 2 + pa0));
            c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
            s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
        }
        if (rb) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(cs + pb0));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(cs + p.rotary_dim / 2 + pb0));
            c[4] = x.x, c[5] = x.y, c[6] = x.z, c[7] = x.w;
            s[4] = y.x, s[5] = y.y, s[6] = y.z, s[7] = y.w;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int seg = seg0 + u * GPW;
            const bool on = seg < segs;
            const bool is_q = seg < p.q_segs;
            const bool is_v = seg >= p.q_segs + p.k_segs;
            const T *w = static_cast<const T *>(is_q ? p.q_norm : p.k_norm);
            float x[16];
            if (on) {
                widen8<T>(xa[u], x);
                widen8<T>(xb[u], x + 8);
            }
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ss = on ? fmaf(x[i], x[i], ss) : 0.f;
#pragma unroll
            for (int o = 1; o < TS; o <<= 1)
                ss += __shfl_xor_sync(FULL, ss, o);
            if (!on)
                continue;
            if (!is_v) {
                if (w) {
                    const float inv = rsqrtf(ss * (1.f / d) + p.eps);
                    float wf[16];
                    widen8<T>(__ldg(reinterpret_cast<const uint4 *>(w) + va), wf);
                    widen8<T>(__ldg(reinterpret_cast<const uint4 *>(w) + vb), wf + 8);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[i] *= inv * wf[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // pair i of the lane: half-split (x[i], x[8 + i]); interleaved
                    // (x[2i], x[2i + 1])
                    float &a = INTER ? x[2 * i] : x[i];
                    float &b = INTER ? x[2 * i + 1] : x[8 + i];
                    const float ra_ = a * c[i] - b * s[i], rb_ = b * c[i] + a * s[i];
                    const bool turn = INTER ? (i < 4 ? ra : rb) : ra;
                    a = turn ? ra_ : a;
                    b = turn ? rb_ : b;
                }
                xa[u] = narrow8<T>(x);
                xb[u] = narrow8<T>(x + 8);
            }
            T *dst;
            if (is_q) {
                dst = static_cast<T *>(p.q_out) + tok * p.q_out_stride + seg * d;
            } else {
                const int j = seg - p.q_segs - (is_v ? p.k_segs : 0);
                if (p.slots) {
                    const long long blk = slot / kBlockSize, off = slot % kBlockSize;
                    const int head = j / p.num_maps, part = j - head * p.num_maps;
                    dst = static_cast<T *>(is_v ? p.v_cache : p.k_cache) +
                          ((blk * p.num_kv_heads + head) * kBlockSize + off) *
                              (long long)(p.num_maps * d) +
                          part * d;
                } else {
                    dst = static_cast<T *>(p.k_out) + tok * p.k_out_stride + j * d;
                }
            }
            reinterpret_cast<uint4 *>(dst)[is_v ? t : va] = xa[u];
            reinterpret_cast<uint4 *>(dst)[is_v ? t + TS : vb] = xb[u];
        }
    }
}

template <typename T, int TS, bool INTER>
const void *pick()
{
    return reinterpret_cast<const void *>(&rope_kernel_t<T, TS, INTER, 1>);
}

template <typename T>
const void *pick_t(int ts, bool inter)
{
    switch (ts) {
    case 2:
        return inter ? pick<T, 2, true>() : pick<T, 2, false>();
    case 4:
        return inter ? pick<T, 4, true>() : pick<T, 4, false>();
    default:
        return inter ? pick<T, 8, true>() : pick<T, 8, false>();
    }
}

}  // namespace

RopeKernel rope_kernel(const RopeParams &p, bool bf16, int head_dim, bool interleaved, int num_sms)
{
    const int ts = head_dim / p.num_maps / 16;
    const int gpw = 32 / ts;
    const long long segs = (long long)p.q_segs + p.k_segs + p.v_segs;
    const long long units = (segs + gpw - 1) / gpw * p.num_tokens;
    RopeKernel r{};
    if (units >= (1LL << 31))
        return r;
    r.fn = bf16 ? pick_t<__nv_bfloat16>(ts, interleaved) : pick_t<__half>(ts, interleaved);
    r.threads = kRopeThreads;
    const long long need = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    const long long cap = (long long)num_sms * 8;
    r.blocks = (int)(need < cap ? need : cap);
    return r;
}

}  // namespace pa
