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
// Every element is read once and written once, so HBM bounds a large call (and
// the launch a decode step's few tokens); behind HBM, instruction issue: packed
// two-wide fp32 arithmetic, angles once per unit of work and weights once per
// warp took 32768 tokens of 32/8 heads x 128 from 155 to 135 us, the rings and
// the split of rope_many_kernel to 127 us, 95 % of the measured copy rate.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_rope.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
// Rounds of a unit, at most: in registers, and through the rings, whose two
// stages a warp hold as many bytes as three of four rounds (32768 tokens without
// the pool write 127.4 us against 130.2, 16384 with it 66.5 against 69.7: fewer
// units, each with its own angles and copies)
constexpr int kFewRounds = 4;
constexpr int kManyRounds = 6;
constexpr int kRopeStages = 2;     // units in flight per warp

// eight 16-bit channels as four packed pairs of fp32, and back
template <typename T>
__device__ __forceinline__ void widen8(const uint4 &v, uint64_t *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Elem<T>::to_f2(w[i]);
        x[i] = f2_pack(f.x, f.y);
    }
}

template <typename T>
__device__ __forceinline__ uint4 narrow8(const uint64_t *x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(x[i], a, b);
        w[i] = Mma<T>::pack(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint64_t f2_swap(uint64_t x)
{
    float a, b;
    f2_unpack(x, a, b);
    return f2_pack(b, a);
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t f2_neg(uint64_t x)
{
    return x ^ 0x8000000080000000ull;
}

// What a lane's rotations take from a token's table row, packed as its channels
// are.  Half-split: cosines and sines of its eight pairs.  Interleaved: of four
// pairs of each vector, (cos, cos) and (-sin, sin) for a pair's two channels.
template <bool INTER>
struct RopeAngles {
    uint64_t c[INTER ? 8 : 4], s[INTER ? 8 : 4];
    uint64_t n[INTER ? 1 : 4];                // half-split: -s
};

// A lane's part of the work, the same in both kernels below.  A warp takes a
// unit: `iters` rounds of 32 / TS consecutive segments of one token's [q | k | v]
// list, TS = d / 16 lanes a segment.  A lane owns two 16-byte vectors of its
// segment, placed so that it holds both channels of every pair it rotates:
// vectors (t, t + rotary_dim / 16) half-split, any two when interleaved.  So a
// rotation needs no data from another lane, and a lane reads and writes the
// same elements only (q_out may be q).  The lane's channels are the same in
// every segment: its weights stay in registers, its angles for a unit.
template <typename T, int TS, bool INTER>
struct RopeLane {
    static constexpr int GPW = 32 / TS;       // segments of a round
    static constexpr int d = 16 * TS;
    int t, grp;                               // lane within its segment, segment within the round
    int va, vb;                               // its vectors of a q or k segment (v: t and t + TS)
    bool ra, rb;                              // whether they are rotated
    int k0, v0, segs;                         // first k and v segments of the list, its length
    uint64_t qw[8], kw[8];                    // its channels' norm weights

    __device__ __forceinline__ explicit RopeLane(const RopeParams &p)
    {
        const int lane = threadIdx.x & 31, rot16 = p.rotary_dim / 16;
        t = lane % TS;
        grp = lane / TS;
        va = t;
        vb = t + TS;
        if constexpr (!INTER) {
            // lanes past the rotated channels take the vectors left over, two each
            va = t < rot16 ? t : 2 * t;
            vb = t < rot16 ? t + rot16 : 2 * t + 1;
        }
        ra = INTER ? va < 2 * rot16 : t < rot16;
        rb = INTER ? vb < 2 * rot16 : t < rot16;
        k0 = p.q_segs;
        v0 = k0 + p.k_segs;
        segs = v0 + p.v_segs;
    }

    __device__ __forceinline__ void load_weights(const RopeParams &p)
    {
        weights(qw, p.q_norm);
        weights(kw, p.k_norm);
    }

    __device__ __forceinline__ void weights(uint64_t (&w)[8], const void *from) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = f2_pack(1.f, 1.f);
        if (from) {
            widen8<T>(__ldg(static_cast<const uint4 *>(from) + va), w);
            widen8<T>(__ldg(static_cast<const uint4 *>(from) + vb), w + 4);
        }
    }

    __device__ __forceinline__ void angles(const RopeParams &p, const float *cs,
                                           RopeAngles<INTER> &g) const
    {
        const float *sn = cs + p.rotary_dim / 2;
        const int pa0 = INTER ? 4 * va : 8 * t, pb0 = INTER ? 4 * vb : 8 * t + 4;
        float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 z = x, w = y;
        if (ra) {
            x = *reinterpret_cast<const float4 *>(cs + pa0);
            y = *reinterpret_cast<const float4 *>(sn + pa0);
        }
        if (rb) {
            z = *reinterpret_cast<const float4 *>(cs + pb0);
            w = *reinterpret_cast<const float4 *>(sn + pb0);
        }
        if constexpr (INTER) {
            const float c[8] = {x.x, x.y, x.z, x.w, z.x, z.y, z.z, z.w};
            const float s[8] = {y.x, y.y, y.z, y.w, w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g.c[i] = f2_pack(c[i], c[i]);
                g.s[i] = f2_pack(-s[i], s[i]);
            }
        } else {
            g.c[0] = f2_pack(x.x, x.y), g.c[1] = f2_pack(x.z, x.w);
            g.c[2] = f2_pack(z.x, z.y), g.c[3] = f2_pack(z.z, z.w);
            g.s[0] = f2_pack(y.x, y.y), g.s[1] = f2_pack(y.z, y.w);
            g.s[2] = f2_pack(w.x, w.y), g.s[3] = f2_pack(w.z, w.w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                g.n[i] = f2_neg(g.s[i]);
        }
    }

    // 1 / sqrt(mean x^2 + eps) of the lane's segment; every lane takes part.
    __device__ __forceinline__ float inverse_rms(const RopeParams &p, const uint64_t (&x)[8]) const
    {
        uint64_t s0 = f2_mul(x[0], x[0]), s1 = f2_mul(x[4], x[4]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            s0 = f2_fma(x[i], x[i], s0);
            s1 = f2_fma(x[4 + i], x[4 + i], s1);
        }
        float lo, hi;
        f2_unpack(f2_add(s0, s1), lo, hi);
        float ss = lo + hi;
#pragma unroll
        for (int o = 1; o < TS; o <<= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        return rsqrtf(fmaf(ss, 1.f / d, p.eps));
    }

    __device__ __forceinline__ void rotate(uint64_t (&x)[8], const RopeAngles<INTER> &g) const
    {
        if constexpr (INTER) {
            if (ra) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = f2_fma(f2_swap(x[i]), g.s[i], f2_mul(x[i], g.c[i]));
            }
            if (rb) {
#pragma unroll
                for (int i = 4; i < 8; ++i)
                    x[i] = f2_fma(f2_swap(x[i]), g.s[i], f2_mul(x[i], g.c[i]));
            }
        } else if (ra) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t a = x[i], b = x[4 + i];
                x[i] = f2_fma(a, g.c[i], f2_mul(b, g.n[i]));
                x[4 + i] = f2_fma(b, g.c[i], f2_mul(a, g.s[i]));
            }
        }
    }

    // A round whose segments are all q, or all k: w and `norm` are theirs.
    __device__ __forceinline__ void turn(const RopeParams &p, const uint64_t (&w)[8], bool norm,
                                         const RopeAngles<INTER> &g, uint4 &xa, uint4 &xb) const
    {
        uint64_t x[8];
        widen8<T>(xa, x);
        widen8<T>(xb, x + 4);
        if (norm) {
            const float inv = inverse_rms(p, x);
            const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = f2_mul(x[i], f2_mul(w[i], inv2));
        }
        rotate(x, g);
        xa = narrow8<T>(x);
        xb = narrow8<T>(x + 4);
    }

    // A round of any segments: the lane's is `seg`, a value segment (or none)
    // where it is not below v0.
    __device__ __forceinline__ void turn_mixed(const RopeParams &p, int seg,
                                               const RopeAngles<INTER> &g, uint4 &xa,
                                               uint4 &xb) const
    {
        const bool is_k = seg >= k0, norm = is_k ? p.k_norm != nullptr : p.q_norm != nullptr;
        uint64_t x[8];
        widen8<T>(xa, x);
        widen8<T>(xb, x + 4);
        const float inv = inverse_rms(p, x);
        if (seg >= v0)
            return;
        if (norm) {
            const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = f2_mul(x[i], f2_mul(is_k ? kw[i] : qw[i], inv2));
        }
        rotate(x, g);
        xa = narrow8<T>(x);
        xb = narrow8<T>(x + 4);
    }

    // Where a token's rows go: q_out, and k_out or the pools' slot.
    struct Target {
        T *q, *k, *kc, *vc;
    };
    __device__ __forceinline__ Target target(const RopeParams &p, unsigned tok, int64_t slot) const
    {
        Target to{};
        to.q = static_cast<T *>(p.q_out) + tok * p.q_out_stride;
        if (p.slots) {
            const long long at = (slot / kBlockSize * p.num_kv_heads * kBlockSize +
                                  slot % kBlockSize) * (long long)(p.num_maps * d);
            to.kc = static_cast<T *>(p.k_cache) + at;
            to.vc = static_cast<T *>(p.v_cache) + at;
        } else {
            to.k = static_cast<T *>(p.k_out) + tok * p.k_out_stride;
        }
        return to;
    }

    // Segment j of the keys or values in a pool: part j % num_maps of head
    // j / num_maps, whose rows lie 16 tokens apart.
    __device__ __forceinline__ int pool_offset(const RopeParams &p, int j) const
    {
        return p.num_maps == 2 ? ((j >> 1) * (2 * kBlockSize) + (j & 1)) * d : j * (kBlockSize * d);
    }

    __device__ __forceinline__ void put(T *row, int a, int b, const uint4 &xa,
                                        const uint4 &xb) const
    {
        reinterpret_cast<uint4 *>(row)[a] = xa;
        reinterpret_cast<uint4 *>(row)[b] = xb;
    }

    // Turns and stores one round, first .. first + GPW - 1, of which segments
    // below `end` are the unit's; xa, xb are the lane's vectors of it.
    __device__ __forceinline__ void round(const RopeParams &p, const Target &to, int first, int end,
                                          const RopeAngles<INTER> &g, uint4 &xa, uint4 &xb) const
    {
        const int seg = first + grp;
        if (first + GPW <= min(end, k0)) {
            turn(p, qw, p.q_norm != nullptr, g, xa, xb);
            put(to.q + seg * d, va, vb, xa, xb);
        } else if (first >= k0 && first + GPW <= min(end, v0)) {
            turn(p, kw, p.k_norm != nullptr, g, xa, xb);
            put(p.slots ? to.kc + pool_offset(p, seg - k0) : to.k + (seg - k0) * d, va, vb, xa, xb);
        } else {
            if (first < v0)
                turn_mixed(p, seg, g, xa, xb);
            if (seg >= end)
                return;
            if (seg < k0)
                put(to.q + seg * d, va, vb, xa, xb);
            else if (seg >= v0)
                put(to.vc + pool_offset(p, seg - v0), t, t + TS, xa, xb);
            else
                put(p.slots ? to.kc + pool_offset(p, seg - k0) : to.k + (seg - k0) * d, va, vb, xa,
                    xb);
        }
    }
};

// Whether a token is written at all: padding is not, and a bad position or slot
// is reported (by the caller that passes `report`) and skipped.
__device__ __forceinline__ bool rope_live(const RopeParams &p, int pos, int64_t slot, bool report)
{
    if (pos < 0 || slot < 0)
        return false;
    if (pos >= p.max_position) {
        if (report)
            record_error(p.err, PA_DEVERR_POSITION_RANGE);
        return false;
    }
    if (p.slots && slot >= p.num_slots) {
        if (report)
            record_error(p.err, PA_DEVERR_SLOT_RANGE);
        return false;
    }
    return true;
}

// Few units: a warp takes at most one, its rows straight into registers.
template <typename T, int TS, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2)
rope_few_kernel(const RopeParams p, const int iters)
{
    constexpr int U = kFewRounds;
    using Lane = RopeLane<T, TS, INTER>;
    constexpr int d = Lane::d, GPW = Lane::GPW;
    grid_dependents_launch();
    grid_dependency_wait();
    Lane me(p);
    const int per_unit = iters * GPW;
    const unsigned chunks = (unsigned)(me.segs + per_unit - 1) / per_unit;
    const unsigned unit = blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32;
    const unsigned tok = unit / chunks;
    if (tok >= (unsigned)p.num_tokens)
        return;
    const int begin = (int)(unit - tok * chunks) * per_unit;
    const int end = min(me.segs, begin + per_unit);
    const T *qrow = static_cast<const T *>(p.q) + tok * p.q_stride;
    const T *krow = static_cast<const T *>(p.k) + tok * p.k_stride - (long long)me.k0 * d;
    const T *vrow = static_cast<const T *>(p.v) + tok * p.v_stride - (long long)me.v0 * d;
    // the rows' loads go out before the token's position and slot are known
    uint4 xa[U], xb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int seg = begin + u * GPW + me.grp;
        xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
        if (seg < end) {
            const bool is_v = seg >= me.v0;
            const uint4 *row = reinterpret_cast<const uint4 *>(
                (seg < me.k0 ? qrow : is_v ? vrow : krow) + seg * d);
            xa[u] = row[is_v ? me.t : me.va];
            xb[u] = row[is_v ? me.t + TS : me.vb];
        }
    }
    const int pos = __ldg(p.positions + tok);
    const int64_t slot = p.slots ? __ldg(p.slots + tok) : 0;
    me.load_weights(p);
    if (!rope_live(p, pos, slot, begin == 0 && (threadIdx.x & 31) == 0))
        return;                               // the same for the whole warp
    RopeAngles<INTER> g;
    me.angles(p, p.cos_sin + (long long)pos * p.rotary_dim, g);
    const typename Lane::Target to = me.target(p, tok, slot);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int first = begin + u * GPW;
        if (first >= end)
            break;                            // the same for the whole warp
        me.round(p, to, first, end, g, xa[u], xb[u]);
    }
}

// Many units: every warp walks units a fixed step apart, each unit's rows and
// table row copied by bulk copies into the warp's own ring of shared-memory
// stages, kRopeStages units ahead, about 200 KB in flight an SM.  Warps never
// wait for each other.
struct RopeStage {
    static constexpr int kRows = kManyRounds * 1024;   // a round is 32 lanes x 32 bytes
    static constexpr int kTable = 512;                 // a table row of at most 128 floats
    static constexpr int kBytes = kRows + kTable;
};

template <typename T, int TS, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2)
rope_many_kernel(const RopeParams p, const int iters, const RopeSplit split)
{
    using Lane = RopeLane<T, TS, INTER>;
    constexpr int d = Lane::d, GPW = Lane::GPW, S = kRopeStages, W = kRopeThreads / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[W * S];
    __shared__ int64_t slot_of[W * S];        // of the stage's token; -1: not written
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    unsigned char *ring = smem + (size_t)warp * S * RopeStage::kBytes;
    const uint32_t bar0 = smem_addr(&bars[warp * S]);
    if (lane == 0) {
        for (int i = 0; i < S; ++i)
            mbar_init(bar0 + 8 * i, 1);
        mbar_init_fence();
    }
    __syncwarp();
    grid_dependents_launch();
    grid_dependency_wait();
    Lane me(p);
    me.load_weights(p);
    const int per_unit = iters * GPW;
    const unsigned chunks = (unsigned)(me.segs + per_unit - 1) / per_unit;
    // this warp's units: begin, begin + step, .. below end
    unsigned units = chunks * (unsigned)p.num_tokens, warps, unit0;
    if (blockIdx.x < split.long_blocks) {
        unit0 = blockIdx.x * W + warp;
        warps = split.long_blocks * W;
        units = min(units, split.long_units);
    } else {
        const unsigned at = split.long_units + (blockIdx.x - split.long_blocks) * split.short_units;
        unit0 = at + warp;
        warps = W;
        units = min(units, at + split.short_units);
    }
    const uint64_t pol = l2_evict_first_policy();      // rows are read once

    // lane 0's side: the next unit to copy, its position and slot already loaded
    unsigned next = unit0;
    int npos = 0;
    int64_t nslot = 0;
    auto peek = [&]() {
        if (lane == 0 && next < units) {
            npos = __ldg(p.positions + next / chunks);
            nslot = p.slots ? __ldg(p.slots + next / chunks) : 0;
        }
    };
    auto issue = [&](int st) {
        if (lane == 0 && next < units) {
            const unsigned tok = next / chunks;
            const int begin = (int)(next - tok * chunks) * per_unit;
            const int end = min(me.segs, begin + per_unit);
            const bool live = rope_live(p, npos, nslot, begin == 0);
            slot_of[warp * S + st] = live ? nslot : -1;
            const uint32_t bar = bar0 + 8 * st;
            if (!live) {
                mbar_arrive(bar);
            } else {
                const uint32_t dst = smem_addr(ring + st * RopeStage::kBytes);
                mbar_arrive_expect_tx(bar, (uint32_t)((end - begin) * d * 2 + p.rotary_dim * 4));
                auto part = [&](const void *base, long long stride, int lo, int hi) {
                    const int a = max(begin, lo), b = min(end, hi);
                    if (a < b)
                        bulk_load(dst + (a - begin) * d * 2,
                                  static_cast<const T *>(base) + tok * stride +
                                      (long long)(a - lo) * d,
                                  (b - a) * d * 2, bar, pol);
                };
                part(p.q, p.q_stride, 0, me.k0);
                part(p.k, p.k_stride, me.k0, me.v0);
                part(p.v, p.v_stride, me.v0, me.segs);
                bulk_load(dst + RopeStage::kRows, p.cos_sin + (long long)npos * p.rotary_dim,
                          p.rotary_dim * 4, bar);
            }
        }
        next += warps;
        peek();
    };
    peek();
#pragma unroll 1
    for (int st = 0; st < S; ++st)
        issue(st);

    unsigned it = 0;
    for (unsigned unit = unit0; unit < units; unit += warps, ++it) {
        const int st = it % S;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + 8 * st, (it / S) & 1))) {
            // a copy that takes a second: report it, let the others land (each
            // wait bounded) and stop
            if (lane == 0)
                record_error(p.err, PA_DEVERR_TIMEOUT);
            for (unsigned x = it; x < it + S && unit0 + x * warps < units; ++x)
                mbar_wait_bounded(bar0 + 8 * (x % S), (x / S) & 1);
            break;
        }
        const int64_t slot = slot_of[warp * S + st];
        if (slot >= 0) {                      // the same for the whole warp
            const unsigned tok = unit / chunks;
            const int begin = (int)(unit - tok * chunks) * per_unit;
            const int end = min(me.segs, begin + per_unit);
            const unsigned char *stage = ring + st * RopeStage::kBytes;
            RopeAngles<INTER> g;
            me.angles(p, reinterpret_cast<const float *>(stage + RopeStage::kRows), g);
            const typename Lane::Target to = me.target(p, tok, slot);
            int first = begin;
            // the rounds that hold queries alone, by far the most, without the
            // choices of round() (4096 tokens 21.8 -> 20.5 us; 32768, where HBM is
            // the bound, 126.7 -> 127.5)
            const int qend = min(end, me.k0) - GPW;
            const unsigned char *from = stage + me.grp * (d * 2);
            T *dst = to.q + (begin + me.grp) * d;
#pragma unroll 3
            for (; first <= qend; first += GPW) {
                uint4 xa = reinterpret_cast<const uint4 *>(from)[me.va];
                uint4 xb = reinterpret_cast<const uint4 *>(from)[me.vb];
                me.turn(p, me.qw, p.q_norm != nullptr, g, xa, xb);
                me.put(dst, me.va, me.vb, xa, xb);
                from += GPW * d * 2;
                dst += GPW * d;
            }
#pragma unroll 1
            for (; first < end; first += GPW) {
                const int seg = first + me.grp;
                uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa;
                if (seg < end) {
                    const bool is_v = seg >= me.v0;
                    const uint4 *row =
                        reinterpret_cast<const uint4 *>(stage + (seg - begin) * d * 2);
                    xa = row[is_v ? me.t : me.va];
                    xb = row[is_v ? me.t + TS : me.vb];
                }
                me.round(p, to, first, end, g, xa, xb);
            }
        }
        __syncwarp();                         // the stage is read: copy into it again
        issue(st);
    }
}

template <typename T, int TS, bool INTER>
void pick(RopeKernel *r, bool many)
{
    r->fn = many ? reinterpret_cast<const void *>(&rope_many_kernel<T, TS, INTER>)
                 : reinterpret_cast<const void *>(&rope_few_kernel<T, TS, INTER>);
}

template <typename T>
void pick(RopeKernel *r, int ts, bool inter, bool many)
{
    switch (ts) {
    case 2:
        return inter ? pick<T, 2, true>(r, many) : pick<T, 2, false>(r, many);
    case 4:
        return inter ? pick<T, 4, true>(r, many) : pick<T, 4, false>(r, many);
    default:
        return inter ? pick<T, 8, true>(r, many) : pick<T, 8, false>(r, many);
    }
}

}  // namespace

RopeKernel rope_kernel(const RopeParams &p, bool bf16, int head_dim, bool interleaved, int num_sms)
{
    constexpr int W = kRopeThreads / 32;
    const int ts = head_dim / p.num_maps / 16;
    const int gpw = 32 / ts;
    const long long segs = (long long)p.q_segs + p.k_segs + p.v_segs;
    const long long rounds = (segs + gpw - 1) / gpw;
    const long long resident = 2LL * W * num_sms;      // warps of one wave
    RopeKernel r{};
    // units of at most `most` rounds, of fewer where that would leave SMs without
    // warps
    auto cut = [&](int most) {
        long long chunks = (rounds + most - 1) / most;
        chunks = std::max(chunks, std::min(rounds, resident / p.num_tokens));
        r.iters = (int)((rounds + chunks - 1) / chunks);
        return (rounds + r.iters - 1) / r.iters * p.num_tokens;
    };
    long long units = cut(kFewRounds);
    // Few units go one to a warp, rows into registers; from three a warp on,
    // through the rings.  Measured (32/8 heads x 128, bf16, pool write, in a
    // graph): 1536 tokens 9.8 us against 11.9 through the rings, 2048 13.1
    // against 13.5, 2560 16.0 against 14.7, 4096 21.8 against 19.9.
    const bool many = units > 3 * resident;
    if (many)
        units = cut(kManyRounds);
    if (units >= (1LL << 31))
        return r;
    bf16 ? pick<__nv_bfloat16>(&r, ts, interleaved, many) : pick<__half>(&r, ts, interleaved, many);
    r.threads = kRopeThreads;
    r.blocks = (int)((units + W - 1) / W);
    if (!many)
        return r;
    // One wave of blocks takes an even share each, then blocks of one unit a
    // warp the remainder.  With many units a warp the SMs drift apart (13 % of
    // their time idle at 40 units of four rounds), so a tenth is left to blocks of
    // two units a warp, which the hardware hands out as SMs come free.  With the
    // pool write 32768 tokens (27 units a warp) 127.4 us against 136.7, 16384
    // 66.0 against 71.0, 8192 (6.7 units) 36.1 against 34.6; without it 107.0
    // against 115.6, 55.0 against 58.2, and 6000 tokens (4.9) 24.3 against 23.1.
    const long long each = units / resident;
    const bool spare = each >= 12;
    const long long tail = W * (spare ? 2 : 1);
    r.split.long_blocks = 2 * num_sms;
    r.split.long_units = (unsigned)((spare ? each - each / 10 : each) * resident);
    r.split.short_units = (unsigned)tail;
    r.blocks = r.split.long_blocks + (int)((units - r.split.long_units + tail - 1) / tail);
    r.smem = (size_t)W * kRopeStages * RopeStage::kBytes;
    return r;
}

}  // namespace pa
