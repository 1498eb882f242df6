// pa_mass.cu -- accumulated attention weight (sm_103a): how much softmax
// weight each token of a sequence has been given, summed over queries and the
// heads of a group.
//
//     mass[s][h][t] = decay * mass[s][h][t] + sum_{i, g} p_ig(t),
//     p_ig(t) = 2^(x_ig(t) - m_ig) / l_ig,  x the scaled scores in base 2
//
// A column sum of a softmax needs every row's maximum and sum before the first
// term can be added, so the scores are either kept (a decode: 4 bytes a score
// beside 4 head_dim bytes of K/V for the token and kv head) or computed twice (a
// chunk of queries, whose scores would outweigh the keys).
#include <cuda.h>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_mass.h"
#include "pa_ragged.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

// One token's new mass; a token of this call (fresh) has none from before.
__device__ __forceinline__ float add_mass(float *at, float decay, bool fresh, float sum)
{
    return fresh || decay == 0.f ? sum : fmaf(*at, decay, sum);
}

// ---------------------------------------------------------------------------
// After a decode: every token's weights from the kept scores.  A warp takes 128
// tokens of a (sequence, kv head), four a lane a stride of 32 apart.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kMassFinishThreads)
decode_mass_finish_kernel(const DecodeMassParams p)
{
    constexpr int NTH = kMassFinishThreads, TOK = 128;
    __shared__ RaggedSmem sm;
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (NTH / 32), me = blockIdx.x * (NTH / 32) + (threadIdx.x >> 5);
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv, cols = score_cols(G);
    const int T = p.max_blocks * kBlockSize;
    grid_dependents_launch();
    grid_dependency_wait();
    for (int begin = 0; begin < p.num_seqs; begin += kRaggedSeqs) {
        const int n = min(kRaggedSeqs, p.num_seqs - begin);
        ragged_prefix<NTH>(sm, begin, n, [&](int s) {
            const int L = min(max(__ldg(p.seq_lens + s), 0), T);   // (the decode has reported it)
            return (L + TOK - 1) / TOK;
        });
        const long long total = (long long)sm.pre[n] * Hkv;
        for (long long u = me; u < total; u += warps) {
            const int i = ragged_find(sm, n, (int)(u / Hkv));
            const int nt = sm.pre[i + 1] - sm.pre[i];
            const int at = (int)(u - (long long)sm.pre[i] * Hkv);
            const int s = begin + i, h = at / nt, t0 = at % nt * TOK + lane;
            const int L = min(max(__ldg(p.seq_lens + s), 0), T);
            const size_t run = (size_t)s * Hkv + h;
            const float *x = p.scores + (run * T + t0) * cols;
            const float2 *stat = p.stat + (size_t)s * p.num_heads + h * G;
            float *mass = p.mass + run * T + t0;
            // every load of four heads in flight at once, and the old masses with the first
            float old[4], sum[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = t0 + 32 * k;
                old[k] = t < L - 1 && p.decay != 0.f ? __ldcg(mass + 32 * k) : 0.f;
                sum[k] = 0.f;
            }
            for (int g = 0; g < G; g += 4) {
                float2 st[4], y[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st[i] = g + i < G ? __ldcg(stat + g + i) : make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (t0 + 32 * k < L && g + 2 * i < G)
                            y[k][i] = __ldcg(reinterpret_cast<const float2 *>(
                                x + (size_t)32 * k * cols + g + 2 * i));
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (t0 + 32 * k < L && g + 2 * i < G) {
                            sum[k] = fmaf(exp2f(y[k][i].x - st[2 * i].x), st[2 * i].y, sum[k]);
                            if (g + 2 * i + 1 < G)
                                sum[k] = fmaf(exp2f(y[k][i].y - st[2 * i + 1].x), st[2 * i + 1].y,
                                              sum[k]);
                        }
            }
            // (the newest token has no mass from before: old is 0)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t0 + 32 * k < L)
                    mass[32 * k] = fmaf(old[k], p.decay, sum[k]);
        }
    }
}

// ---------------------------------------------------------------------------
// A chunk of queries, on the fifth-generation tensor cores.  A unit of work is
// 2 x 128 (token, head) rows of a (sequence, kv head); they stay in shared
// memory while the sequence's keys stream past in 128-key tiles (TMA, a ring of
// slots), a part of them per thread block.  Pass 1 (SUMS false) takes
// S = Q.K^T, a thread a query row, and leaves each row's maximum and sum over its
// part; pass 2 takes S^T = K.Q^T, a thread a key, so that the sum over the
// queries is a sum over the thread's own columns, with the row's statistics read
// from shared memory as a broadcast.  Scores live in tensor memory, two buffers
// a query tile, so the MMAs of the next key tile run while the softmax warps
// read this one.
// ---------------------------------------------------------------------------
template <int D>
struct MassShape {
    static constexpr int BM = kMassRows, NG = kMassTiles, BN = kMassKeys;
    static constexpr int NB = BN / kBlockSize;
    static constexpr int HALVES = D / 64;
    static constexpr int BOX = 2048;                      // 16 rows x 128 B
    static constexpr int Q_BYTES = BM * D * 2;            // [half][128 rows][128 B]
    static constexpr int SLOT_BYTES = BN * D * 2;         // [half][8 blocks][16 rows][128 B]
    static constexpr int NSLOT = D == 128 ? 5 : 8;
    static constexpr int OFF_SLOT = NG * Q_BYTES;
    static constexpr int OFF_LSE = OFF_SLOT + NSLOT * SLOT_BYTES;
    // full[NSLOT] empty[NSLOT] s[NG][2] read[NG][2] q[NG] drain, then TMEM base, abort flag
    static constexpr int NBAR = 2 * NSLOT + 5 * NG + 1;
    static constexpr int OFF_BAR = OFF_LSE + NG * BM * 4;
    static constexpr int SMEM = 1024 + OFF_BAR + NBAR * 8 + 8;
    static constexpr int THREADS = 64 + NG * 128;
    static_assert(SMEM <= 227 * 1024, "one block per SM");
};

__device__ __forceinline__ void group_sync(int grp)
{
    asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
}

template <typename T, int D, bool SUMS>
__global__ void __launch_bounds__(MassShape<D>::THREADS)
prefill_mass_kernel(const PrefillMassParams p, const __grid_constant__ CUtensorMap tmk)
{
    using Sh = MassShape<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int NS = Sh::NSLOT;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_addr(smem), slot_addr = sbase + Sh::OFF_SLOT;
    float *lse = reinterpret_cast<float *>(smem + Sh::OFF_LSE);      // minus the rows' log sums
    const uint32_t bar_addr = sbase + Sh::OFF_BAR;
    auto full_bar = [&](int s) { return bar_addr + 8u * s; };
    auto empty_bar = [&](int s) { return bar_addr + 8u * (NS + s); };
    auto s_bar = [&](int g, int b) { return bar_addr + 8u * (2 * NS + 2 * g + b); };
    auto read_bar = [&](int g, int b) { return bar_addr + 8u * (2 * NS + 4 + 2 * g + b); };
    auto q_bar = [&](int g) { return bar_addr + 8u * (2 * NS + 8 + g); };
    const uint32_t drain_bar = bar_addr + 8u * (2 * NS + 10);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Sh::OFF_BAR + Sh::NBAR * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = p.num_kv_heads, Hq = p.num_heads, G = Hq / Hkv;
    const int TPG = Sh::BM / G, TPB = Sh::NG * TPG;       // chunk tokens of a tile, of a unit
    grid_dependents_launch();
    grid_dependency_wait();
    // blocks of one (sequence, head, part of the keys) lie side by side
    int b = blockIdx.x;
    const int rank = b % p.row_blocks;
    b /= p.row_blocks;
    const int split = b % p.splits;
    b /= p.splits;
    const int h = b % Hkv, s = b / Hkv;
    const int L = __ldg(p.seq_lens + s);
    const int qs = __ldg(p.query_start + s);
    const int c = __ldg(p.query_start + s + 1) - qs;
    const bool reporter = !SUMS && rank == 0 && split == 0 && h == 0 && tid == 0;
    if (L < 0 || L > p.max_blocks * kBlockSize) {
        if (reporter)
            record_error(p.err, PA_DEVERR_SEQLEN_RANGE);
        return;
    }
    if (c < 0 || c > L || qs < 0 || c > p.num_queries - qs || (c + TPB - 1) / TPB > p.row_blocks) {
        if (reporter)
            record_error(p.err, PA_DEVERR_QUERY_RANGE);
        return;
    }
    const int t0 = rank * TPB;
    if (t0 >= c)
        return;
    const int t_end = min(t0 + TPB, c);
    const int ng = t_end - t0 > TPG ? 2 : 1;              // query tiles with rows
    const int base = L - c + t0;                          // position of the unit's first token
    const int nt = (L - c + t_end - 1) / Sh::BN + 1;
    const int j0 = (int)((long long)nt * split / p.splits);
    const int ntl = (int)((long long)nt * (split + 1) / p.splits) - j0;   // this block's tiles
    const int nblk = (L + kBlockSize - 1) / kBlockSize;
    const size_t unit = ((size_t)s * Hkv + h) * p.row_blocks + rank;
    if (ntl == 0) {
        // nothing here: an empty part of every row
        if (!SUMS)
            for (int i = tid; i < Sh::NG * Sh::BM; i += Sh::THREADS)
                p.stats[(unit * p.splits + split) * (Sh::NG * Sh::BM) + i] =
                    make_float2(-INFINITY, 0.f);
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
        }
        for (int g = 0; g < Sh::NG; ++g) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(s_bar(g, i), 1);
                mbar_init(read_bar(g, i), 128);
            }
            mbar_init(q_bar(g), Sh::NG * 128);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_addr(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto give_up = [&]() {
        *abort_flag = 1;
        record_error(p.err, PA_DEVERR_TIMEOUT);
    };

    if (warp == 0) {
        // ---------------- producer: key tiles into the ring ----------------
        // lane l holds the pool row of block NB * win + l of a window of WT tiles; lane 0
        // waits for the slot, lanes (half, block) issue the boxes
        constexpr int NB = Sh::NB, WT = 32 / NB;
        const int32_t *table = p.block_tables + (size_t)s * p.max_blocks;
        auto fetch = [&](int w0) {
            const int lb = NB * w0 + lane;
            return lb < nblk ? __ldg(table + lb) : 0;
        };
        auto to_row = [&](int w0, int phys) {
            if (NB * w0 + lane >= nblk)
                return -1;
            if ((unsigned)phys >= (unsigned)p.num_blocks) {
                record_error(p.err, PA_DEVERR_TABLE_RANGE);
                phys = 0;
            }
            return (phys * Hkv + h) * kBlockSize;
        };
        int win = j0;
        int cur = to_row(j0, fetch(j0));
        int nxt = fetch(j0 + WT);
        int last = -1;
        for (int i = 0; i < ntl; ++i) {
            const int j = j0 + i, sl = i % NS;
            if (j == win + WT) {
                win += WT;
                cur = to_row(win, nxt);
                nxt = fetch(win + WT);
            }
            bool ready = true;
            if (lane == 0)
                ready = !*abort_flag &&
                        (i < NS || mbar_wait_bounded(empty_bar(sl), ((i / NS) - 1) & 1));
            if (!__shfl_sync(FULL, ready, 0)) {
                if (lane == 0 && !*abort_flag)
                    give_up();
                break;
            }
            const int nv = min(NB, nblk - NB * j);
            if (lane == 0)
                mbar_arrive_expect_tx(full_bar(sl), (uint32_t)(nv * Sh::HALVES * Sh::BOX));
            const int bb = lane % NB, hf = lane / NB;
            const int row = __shfl_sync(FULL, cur, NB * (j - win) + bb);
            __syncwarp();
            if (hf < Sh::HALVES && row >= 0)
                tma_load_2d(slot_addr + sl * Sh::SLOT_BYTES + (hf * NB + bb) * Sh::BOX, &tmk,
                            64 * hf, row, full_bar(sl));
            if (lane == sl)
                last = i;
        }
        // every issued copy lands before the block may exit
        if (lane < NS && last >= 0 && !mbar_wait_bounded(full_bar(lane), (last / NS) & 1))
            give_up();
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t id = tc::idesc_f16(kBf16, 128, 128, false, false);
        const uint64_t q_desc = tc::sdesc_sw128(sbase, 16, 1024);
        const uint64_t k_desc = tc::sdesc_sw128(slot_addr, 16, 1024);
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(FULL, mbar_wait_bounded(bar, parity));
        };
        bool ok = true;
        for (int i = 0; ok && i < ntl; ++i) {
            const int sl = i % NS, buf = i & 1;
            if (__any_sync(FULL, *abort_flag != 0)) {
                ok = false;
                break;
            }
            for (int g = 0; ok && g < ng; ++g) {
                if (i == 0)
                    ok = wait_all(q_bar(g), 0);
                if (ok && i >= 2)                        // the tile two before has been read
                    ok = wait_all(read_bar(g, buf), ((i >> 1) - 1) & 1);
                ok = ok && wait_all(full_bar(sl), (i / NS) & 1);
                if (!ok)
                    break;
                tc::fence_after_sync();
                const uint64_t qd = q_desc + (uint64_t)((g * Sh::Q_BYTES) >> 4);
                const uint64_t kd = k_desc + (uint64_t)((sl * Sh::SLOT_BYTES) >> 4);
                const uint32_t d = tmem + g * 256 + buf * 128;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t ko = (uint64_t)(((k & 3) * 32 + (k >> 2) * (128 * 128)) >> 4);
                    if (SUMS)
                        tc::mma_ss_warp(d, kd + ko, qd + ko, id, k > 0);
                    else
                        tc::mma_ss_warp(d, qd + ko, kd + ko, id, k > 0);
                }
                tc::commit_warp(s_bar(g, buf));
                if (g == ng - 1)
                    tc::commit_warp(empty_bar(sl));
            }
        }
        if (!ok && lane == 0)
            give_up();
        // no MMA may still run when TMEM is freed
        tc::commit_warp(drain_bar);
        if (!wait_all(drain_bar, 0) && lane == 0)
            give_up();
    } else {
        // ---------------- query rows -> shared memory ----------------
        // K-major, 128-byte swizzle.  Row rr of tile g = (token t0 + g TPG + rr / G, head
        // rr % G); rows past the chunk and those that do not fill a token are zero.
        {
            constexpr int CPR = D / 8, RSTEP = Sh::NG * 128 / CPR;
            constexpr int NPT = Sh::NG * Sh::BM / RSTEP, PER_G = NPT / Sh::NG;
            const T *qg = static_cast<const T *>(p.q);
            const int lt = tid - 64, ch = lt % CPR, hf = ch >> 3, c8 = ch & 7;
            uint4 qv[NPT];
#pragma unroll
            for (int i = 0; i < NPT; ++i) {
                const int r = lt / CPR + i * RSTEP, g = r / Sh::BM, rr = r % Sh::BM;
                const int tok = g * TPG + rr / G, hg = rr % G;
                qv[i] = make_uint4(0, 0, 0, 0);
                if (rr < TPG * G && t0 + tok < c)
                    qv[i] = __ldg(reinterpret_cast<const uint4 *>(
                        qg + ((size_t)(qs + t0 + tok) * Hq + h * G + hg) * D + ch * 8));
            }
#pragma unroll
            for (int i = 0; i < NPT; ++i) {
                const int r = lt / CPR + i * RSTEP, g = r / Sh::BM, rr = r % Sh::BM;
                *reinterpret_cast<uint4 *>(smem + g * Sh::Q_BYTES + hf * (Sh::BM * 128) +
                                           rr * 128 + ((c8 ^ (rr & 7)) << 4)) = qv[i];
                if (i % PER_G == PER_G - 1) {
                    fence_proxy_async_shared();
                    mbar_arrive(q_bar(i / PER_G));
                }
            }
        }
        const int grp = (warp - 2) >> 2;
        const int q4 = warp & 3;                          // TMEM lane quarter of this warp
        const int rr = q4 * 32 + lane;                    // this thread's TMEM lane
        const uint32_t tg = tmem + ((uint32_t)(q4 * 32) << 16) + grp * 256;
        const int tok = grp * TPG + rr / G;
        const bool row_valid = rr < TPG * G && t0 + tok < t_end;
        const float sl2 = p.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        const size_t stat0 = unit * p.splits * (Sh::NG * Sh::BM) + grp * Sh::BM + rr;
        float m = -INFINITY, l = 0.f;
        if (SUMS) {
            // minus log2 of the row's sum over all parts; rows that are none: -inf
            float M = -INFINITY;
            for (int i = 0; i < p.splits; ++i) {
                const float2 a = __ldcg(p.stats + stat0 + (size_t)i * (Sh::NG * Sh::BM));
                const float nM = fmaxf(M, a.x);
                if (nM > -INFINITY)
                    l = l * exp2f(M - nM) + a.y * exp2f(a.x - nM);
                M = nM;
            }
            lse[grp * Sh::BM + rr] = row_valid ? -(M + log2f(l)) : -INFINITY;
            group_sync(grp);
        }
        float *sums = p.sums + (((size_t)s * Hkv + h) * (2 * p.row_blocks) + 2 * rank + grp) *
                                   ((size_t)p.max_blocks * kBlockSize);
        bool ok = true;
        for (int i = 0; grp < ng && i < ntl; ++i) {
            const int buf = i & 1, k0 = (j0 + i) * Sh::BN;
            if (__any_sync(FULL, *abort_flag != 0) ||
                !__all_sync(FULL, mbar_wait_bounded(s_bar(grp, buf), (i >> 1) & 1))) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            uint32_t v[2][64];
            __syncwarp();
            tc::tmem_ld64(tg + buf * 128, v[0]);
            tc::tmem_ld64(tg + buf * 128 + 64, v[1]);
            tc::fence_before_sync();
            mbar_arrive(read_bar(grp, buf));
            float mref = 0.f;
            if (!SUMS) {
                // keys [0, vis] of the tile are visible to this row
                const int vis = row_valid ? base + tok - k0 : -1;
                if (!__all_sync(FULL, vis >= Sh::BN - 1)) {
#pragma unroll
                    for (int e = 0; e < Sh::BN; ++e)
                        if (e > vis)
                            v[e >> 6][e & 63] = __float_as_uint(-INFINITY);
                }
                float mx[8];
#pragma unroll
                for (int a = 0; a < 8; ++a) {
                    auto x = [&](int q) { return __uint_as_float(v[q >> 6][q & 63]); };
                    float t = fmax3(x(a), x(a + 8), x(a + 16));
#pragma unroll
                    for (int q = a + 24; q < 120; q += 16)
                        t = fmax3(t, x(q), x(q + 8));
                    mx[a] = fmaxf(t, x(a + 120));
                }
                const float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                       fmaxf(mx[6], mx[7])) * sl2;    // scale > 0
                if (mt > m) {
                    l *= ex2_approx(m - mt);
                    m = mt;
                }
                mref = m == -INFINITY ? 0.f : m;          // nothing seen yet: weights of zero
            } else {
                // columns [first, 128) of the tile see this key
                const int first = min(max(k0 + rr - base - grp * TPG, 0), 128) * G;
                if (!__all_sync(FULL, first <= 0)) {
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (e < first)
                            v[e >> 6][e & 63] = __float_as_uint(-INFINITY);
                }
            }
            uint64_t sum2[4] = {0, 0, 0, 0};
            const uint64_t nm2 = f2_pack(-mref, -mref);
            const float4 *ls = reinterpret_cast<const float4 *>(lse + grp * Sh::BM);
#pragma unroll
            for (int e = 0; e < 128; e += 4) {
                uint64_t na = nm2, nb = nm2;
                if (SUMS) {
                    const float4 x = ls[e / 4];
                    na = f2_pack(x.x, x.y);
                    nb = f2_pack(x.z, x.w);
                }
                float y0, y1, y2, y3;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e >> 6][e & 63]),
                                         __uint_as_float(v[e >> 6][(e & 63) + 1])), sl2x2, na),
                          y0, y1);
                f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e >> 6][(e & 63) + 2]),
                                         __uint_as_float(v[e >> 6][(e & 63) + 3])), sl2x2, nb),
                          y2, y3);
                sum2[(e >> 2) & 1] =
                    f2_add(sum2[(e >> 2) & 1], f2_pack(ex2_approx(y0), ex2_approx(y1)));
                sum2[2 + ((e >> 2) & 1)] =
                    f2_add(sum2[2 + ((e >> 2) & 1)], f2_pack(ex2_approx(y2), ex2_approx(y3)));
            }
            float a, bsum;
            f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), a, bsum);
            if (!SUMS)
                l += a + bsum;
            else if (k0 + rr < L)
                sums[k0 + rr] = a + bsum;
        }
        if (!ok)
            give_up();
        else if (!SUMS && grp < ng)
            p.stats[stat0 + (size_t)split * (Sh::NG * Sh::BM)] = make_float2(m, l);
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// The sum over a sequence's query tiles, added to the mass: a warp 128 tokens of a
// (sequence, kv head), four a lane.
__global__ void __launch_bounds__(kMassFinishThreads)
prefill_mass_finish_kernel(const PrefillMassParams p)
{
    constexpr int NTH = kMassFinishThreads, TOK = 128;
    __shared__ RaggedSmem sm;
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (NTH / 32), me = blockIdx.x * (NTH / 32) + (threadIdx.x >> 5);
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv, TPG = kMassRows / G;
    const int T = p.max_blocks * kBlockSize;
    grid_dependents_launch();
    grid_dependency_wait();
    for (int begin = 0; begin < p.num_seqs; begin += kRaggedSeqs) {
        const int n = min(kRaggedSeqs, p.num_seqs - begin);
        ragged_prefix<NTH>(sm, begin, n, [&](int s) {
            const int L = __ldg(p.seq_lens + s), qs = __ldg(p.query_start + s);
            const int c = __ldg(p.query_start + s + 1) - qs;
            // what the passes skipped stays as it was
            return L < 0 || L > T || c <= 0 || c > L || qs < 0 || c > p.num_queries - qs ||
                           (c + kMassTiles * TPG - 1) / (kMassTiles * TPG) > p.row_blocks
                       ? 0
                       : (L + TOK - 1) / TOK;
        });
        const long long total = (long long)sm.pre[n] * Hkv;
        for (long long u = me; u < total; u += warps) {
            const int i = ragged_find(sm, n, (int)(u / Hkv));
            const int nt = sm.pre[i + 1] - sm.pre[i];
            const int at = (int)(u - (long long)sm.pre[i] * Hkv);
            const int s = begin + i, h = at / nt, t = at % nt * TOK + 4 * lane;
            const int L = __ldg(p.seq_lens + s);
            const int c = __ldg(p.query_start + s + 1) - __ldg(p.query_start + s);
            if (t >= L)
                continue;
            const size_t run = (size_t)s * Hkv + h;
            const float *part = p.sums + run * (2 * p.row_blocks) * T + t;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            // tiles whose keys reach t (a unit's tiles end where its last row's do)
            const int tiles = (c + TPG - 1) / TPG;
            const int from = max(0, (t - (L - c)) / (kMassTiles * TPG)) * kMassTiles;
#pragma unroll 4
            for (int k = from; k < tiles; ++k) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(part + (size_t)k * T));
                const int end = L - c + min((k / kMassTiles + 1) * kMassTiles * TPG, c);
                sum[0] += x.x;                    // (t itself is reached by the first unit)
                sum[1] += t + 1 < end ? x.y : 0.f;
                sum[2] += t + 2 < end ? x.z : 0.f;
                sum[3] += t + 3 < end ? x.w : 0.f;
            }
            float *mass = p.mass + run * T + t;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t + k < L)
                    mass[k] = add_mass(mass + k, p.decay, t + k >= L - c, sum[k]);
        }
    }
}

template <typename T, int D>
void fill(MassKernels *k)
{
    k->stats = reinterpret_cast<const void *>(&prefill_mass_kernel<T, D, false>);
    k->sums = reinterpret_cast<const void *>(&prefill_mass_kernel<T, D, true>);
    k->threads = MassShape<D>::THREADS;
    k->smem = MassShape<D>::SMEM;
}

}  // namespace

bool prefill_mass_kernels(bool bf16, int head_dim, MassKernels *k)
{
    if (head_dim == 128)
        bf16 ? fill<__nv_bfloat16, 128>(k) : fill<__half, 128>(k);
    else if (head_dim == 64)
        bf16 ? fill<__nv_bfloat16, 64>(k) : fill<__half, 64>(k);
    else
        return false;
    return true;
}

const void *prefill_mass_finish()
{
    return reinterpret_cast<const void *>(&prefill_mass_finish_kernel);
}

const void *decode_mass_finish()
{
    return reinterpret_cast<const void *>(&decode_mass_finish_kernel);
}

}  // namespace pa
