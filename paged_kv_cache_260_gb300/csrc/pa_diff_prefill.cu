// pa_diff_prefill.cu -- chunked prefill of differential attention on the
// fifth-generation tensor cores (tcgen05), over the paged pool.
//
// A head's q row and a token's key row hold two queries and two keys of
// head_dim / 2 channels side by side (map 0, map 1); the values are shared:
//     y = sum_t softmax_t(scale q0.k0_t) v_t - lambda sum_t softmax_t(scale q1.k1_t) v_t
// over the positions a row sees, then an optional RMS norm over head_dim.
//
// One thread block (one per SM) computes 128 rows = (token, q head) pairs of
// one sequence and kv head.  The two maps run side by side on the same Q, K and
// V tiles: per 128-key tile j and map g
//     S_g,j = Q[:, g] . K_j[:, g]^T     (M 128, N 128, K = head_dim / 2)
//     O_g  += P_g,j . V_j               (M 128, N head_dim, K 128)
// so K and V are staged once for both, and O_0, O_1 end up in the same TMEM
// lanes, where the difference is taken.
//
// What bounds it, measured on two 2048-token chunks at 16K (32/8 heads x 128,
// bf16; 1.55 TFLOP): 1400 us, 1.10 PFLOP/s.
//  * A block of 128 rows reads K and V twice as often as the plain prefill's 256
//    rows do: 64 KB a tile, 5.8 TB/s out of L2 over all SMs, the most that any
//    form of this kernel has drawn.  With half of each V tile left out of the
//    copies an earlier form went from 1419 to 1237 us.  The 512 TMEM columns hold
//    two score tiles and two O of 128 columns each, so a block has room for no
//    more rows.  The copies are plain ones, into the block's own shared memory:
//    replicas on several GPUs load this library, and a multicast load must not
//    run there.
//  * Behind that, each map's chain S -> softmax -> P.V -> next S: P lies over score
//    columns, and TMEM has no others.  P.V starts on the first 64 keys while the
//    softmax is at the others; each map has an issuing warp of its own (one for
//    both was busy for 2,300 cycles a tile: every wait on a barrier costs it 100 to
//    250, completed or not); map 1 starts half a tile behind map 0; and as P needs
//    only the second half of the score columns, the next tile's first 64 keys are
//    scored into the first half while the softmax is at its exponentials.
//  * Short contexts (8 x 512 tokens over 0.5K to 4K, 227 us): also a block's start
//    and end, about 11,000 cycles before its first softmax, after its last P and
//    between blocks.  The barriers come first, K_0 and the query rows in flight over
//    the block's last barrier, the norm's weights and lambda are loaded ahead, and
//    output rows are stored by whole lines.
//  * Few query tiles (short chunks against long caches): the SMs without one. A
//    cluster of up to 16 blocks shares the keys of one tile, each block a run of
//    them, and joins its results through distributed shared memory (join_split;
//    128 KB of O, one row in so many to a block; no workspace and no second
//    launch).  16 tokens at 16K, bf16, head_dim 128: 1 x 4/1 heads 208 us on one
//    block, 23 on 16; 2 x 32/8 heads 210, on clusters of 6 46.  As many blocks as
//    let all clusters run at once: with clusters of 8, of which 15 fit, the
//    latter's 16 tiles took 71 us.
//  * P through shared memory, which lets the next S go ahead, costs more shared
//    memory bandwidth than there is; 80-key tiles with P in columns of its own and
//    two threads a row were slower as well.
//
// Warp roles (384 threads):
//   warp 0     TMA producer: K tiles and V tiles through a ring each, K one tile
//              ahead;
//   warps 1-2  issue the MMAs of map 0 and 1 (warp 1 owns the TMEM; the whole warp
//              runs the loop, one elected lane issues);
//   warp 3     warms L2 with the query rows of the block one wave later;
//   warps 4-7 map 0, 8-11 map 1: load the Q tile, then one thread per row (its
//              TMEM lane): scores from TMEM, causal mask, online softmax in base
//              2 with a lazy rescale of O (only when the running maximum grows
//              by more than 2^8), P into TMEM in two halves, rounded to the
//              operand type (the row sum takes the unrounded weights; the product
//              with V needs 16-bit operands, and a second product with what the
//              rounding left over would add a third to the tensor work); at the
//              end each map forms the difference of half of the row's channels.
// TMEM (512 columns): map g has S in [256g, 256g + 128) and O in
// [256g + 128, 256g + 128 + head_dim).  P, packed two per column, overwrites S's
// last 64 columns at head_dim 128, and S_g,j+1 comes in two halves: the first 64
// keys as soon as the softmax has read those of S_g,j, the others after P_g,j . V_j.
// At head_dim 64 P has the map's last 64 columns, and all of S_g,j+1 is issued as
// soon as the softmax has read S_g,j.
// Every wait is bounded; a wait that gives up records PA_DEVERR_TIMEOUT and
// the block drains its copies and MMAs before it frees TMEM and exits.
#include <cuda.h>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_prefill_abi.h"
#include "pa_prefill_plan.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

template <int D>
struct DiffShape {
    static constexpr int BM = kPrefillRows;                 // rows of the block
    static constexpr int BN = kPrefillKeys;                 // keys per tile
    static constexpr int NB = BN / kBlockSize;              // pool blocks per tile
    static constexpr int HALVES = D / 64;                   // 128-byte column boxes
    static constexpr int BOX = 2048;                        // 16 rows x 128 B
    static constexpr int Q_BYTES = BM * D * 2;              // [half][128 rows][128 B]
    static constexpr int SLOT_BYTES = BN * D * 2;           // [half][NB blocks][16 rows][128 B]
    static constexpr int NSLOT = D == 128 ? 3 : 6;          // K slots, and V slots
    static constexpr int OFF_K = Q_BYTES;
    static constexpr int OFF_V = OFF_K + NSLOT * SLOT_BYTES;
    static constexpr int OFF_X = OFF_V + NSLOT * SLOT_BYTES;   // the maps' exchange: [4][128] fp32
    static constexpr int DATA = OFF_X + 4 * BM * 4;
    // kfull, kempty, vfull, vempty [NSLOT]; s, read, o, p low, p high, drain [2];
    // q, z, start; s high [2]; then the TMEM base and the abort flag
    static constexpr int NBAR = 4 * NSLOT + 12 + 3 + 2;
    static constexpr int BAR_BYTES = NBAR * 8 + 8;
    // The operands are aligned up to 1024 bytes inside the dynamic allocation;
    // the barriers sit in whichever end of the 1024-byte slack has room.
    static constexpr int SMEM = DATA + 1024;
    static constexpr int THREADS = 384;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t MAP_COLS = 256;
    static constexpr uint32_t COL_O = 128;
    static constexpr bool SEPARATE_P = COL_O + D + BN / 2 <= MAP_COLS;
    static constexpr uint32_t COL_P = SEPARATE_P ? COL_O + D : BN / 2;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(OFF_K % 1024 == 0 && SLOT_BYTES % 2048 == 0, "swizzle atoms");
    static_assert(BAR_BYTES <= 512, "barriers fit either end of the slack");
    static_assert(SMEM <= 227 * 1024, "one block per SM");
};

// All softmax warps together.
__device__ __forceinline__ void softmax_warps_sync()
{
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

// The pool rows of a run of key tiles, in order: lane l holds the row of block
// NB * win + l of a window of 32 / NB tiles; the next window's table entries are
// already in flight.
template <int NB>
struct TableWindow {
    static constexpr int WT = 32 / NB;
    const PrefillParams &p;
    const int32_t *table;
    int nblk, h, lane, win, cur, nxt;

    // first, second: this lane's entries of the first two windows (fetch)
    __device__ __forceinline__ TableWindow(const PrefillParams &p_, const int32_t *table_, int h_,
                                           int nblk_, int first, int second)
        : p(p_), table(table_), nblk(nblk_), h(h_), lane(threadIdx.x & 31), win(0), nxt(second)
    {
        cur = to_row(0, first);
    }
    // Entry of block NB * w0 + lane, 0 past the sequence.
    static __device__ __forceinline__ int fetch(const int32_t *table, int nblk, int w0)
    {
        const int lb = NB * w0 + (threadIdx.x & 31);
        return lb < nblk ? __ldg(table + lb) : 0;
    }
    __device__ __forceinline__ int to_row(int w0, int phys) const
    {
        if (NB * w0 + lane >= nblk)
            return -1;                  // blocks past the sequence are not loaded
        if ((unsigned)phys >= (unsigned)p.num_blocks) {
            record_error(p.err, PA_DEVERR_TABLE_RANGE);
            phys = 0;
        }
        return (phys * p.num_kv_heads + h) * kBlockSize;
    }
    // Row of this lane's block (lane % NB) of tile j; called for tiles in order.
    __device__ __forceinline__ int row(int j)
    {
        if (j == win + WT) {
            win += WT;
            cur = to_row(win, nxt);
            nxt = fetch(table, nblk, win + WT);
        }
        return __shfl_sync(0xffffffffu, cur, NB * (j - win) + lane % NB);
    }
};

// The blocks of a cluster have each left, for every row of the unit (`rows` of
// them) and map, their keys' maximum and sum (OFF_X: sums, then maxima) and O
// (OFF_K: [map][row][D] fp32, 16-byte chunk i at i ^ (row & 7)).  Block `rank`
// joins the rows rank, rank + SE, ..: 2 SE threads a row, or the power of two
// below.
template <typename T, int D, int SE>
__device__ __forceinline__ void join_split(const PrefillParams &p, uint32_t sbase,
                                           uint32_t abort_addr, int rank, int lt, int rows,
                                           int G, int h, size_t token)
{
    using Sh = DiffShape<D>;
    constexpr int TPR = SE == 3 ? 4 : SE == 6 ? 8 : 2 * SE;
    constexpr int NC = D / 4 < TPR ? 1 : D / 4 / TPR;   // 16-byte chunks of a thread
    static_assert((TPR & (TPR - 1)) == 0 && 256 / TPR * SE >= Sh::BM, "every row has its threads");
    const int row = lt / TPR * SE + rank, tr = lt % TPR;
    const bool live = row < rows && tr < D / 4;
    float y[NC][4], ss = 0.f;
    int aborted = 0;
#pragma unroll
    for (int k = 0; k < NC; ++k)
        y[k][0] = y[k][1] = y[k][2] = y[k][3] = 0.f;
    if (live) {
        // all of a step's loads before the first use: one latency, not one a block
        float f[2][SE], l[2][SE];
#pragma unroll
        for (int c = 0; c < SE; ++c) {
            aborted |= __float_as_int(cluster_load(cluster_addr(abort_addr, c)));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t at = sbase + Sh::OFF_X + (g * Sh::BM + row) * 4;
                l[g][c] = cluster_load(cluster_addr(at, c));
                f[g][c] = cluster_load(cluster_addr(at + 2 * Sh::BM * 4, c));
            }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int c = 0; c < SE; ++c)
                top = fmaxf(top, f[g][c]);
#pragma unroll
            for (int c = 0; c < SE; ++c) {
                f[g][c] = ex2_approx(f[g][c] - top);
                sum = fmaf(l[g][c], f[g][c], sum);
            }
            const float of = (g ? -__ldg(p.lambda + h * G + row % G) : 1.f) / sum;
#pragma unroll
            for (int c = 0; c < SE; ++c)
                f[g][c] *= of;
        }
#pragma unroll
        for (int c = 0; c < SE; ++c) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t at =
                    cluster_addr(sbase + Sh::OFF_K + (g * Sh::BM + row) * (D * 4), c);
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float4 o = cluster_load4(at + (((k * TPR + tr) ^ (row & 7)) << 4));
                    y[k][0] = fmaf(o.x, f[g][c], y[k][0]);
                    y[k][1] = fmaf(o.y, f[g][c], y[k][1]);
                    y[k][2] = fmaf(o.z, f[g][c], y[k][2]);
                    y[k][3] = fmaf(o.w, f[g][c], y[k][3]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < NC; ++k)
            ss += fmaf(y[k][0], y[k][0], y[k][1] * y[k][1]) +
                  fmaf(y[k][2], y[k][2], y[k][3] * y[k][3]);
    }
    __syncwarp();
    float k0 = p.out_scale;
    if (p.norm_w) {
#pragma unroll
        for (int off = 1; off < TPR; off <<= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, off);
        k0 *= rsqrtf(ss * (1.f / D) + p.norm_eps);
    }
    if (!live || aborted)
        return;
    T *out = static_cast<T *>(p.out) +
             ((token + row / G) * p.num_heads + h * G + row % G) * D;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int ch = k * TPR + tr;              // 4 channels
        float w[4] = {k0, k0, k0, k0};
        if (p.norm_w) {
            const uint2 wv = __ldg(static_cast<const uint2 *>(p.norm_w) + ch);
            const float2 a = Elem<T>::to_f2(wv.x), b = Elem<T>::to_f2(wv.y);
            w[0] *= a.x, w[1] *= a.y, w[2] *= b.x, w[3] *= b.y;
        }
        reinterpret_cast<uint2 *>(out)[ch] =
            make_uint2(Mma<T>::pack(y[k][0] * w[0], y[k][1] * w[1]),
                       Mma<T>::pack(y[k][2] * w[2], y[k][3] * w[3]));
    }
}

// one block a query tile, or a cluster of kSplits blocks (by the launch)
template <typename T, int D>
__global__ void __launch_bounds__(DiffShape<D>::THREADS)
diff_prefill_kernel_t(const PrefillParams p, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv)
{
    using Sh = DiffShape<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int NS = Sh::NSLOT;

    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_addr(smem);
    unsigned char *bars = (smem - smem_raw) >= Sh::BAR_BYTES ? smem_raw : smem + Sh::DATA;
    const uint32_t bar_addr = smem_addr(bars);
    auto kfull = [&](int i) { return bar_addr + 8u * i; };
    auto kempty = [&](int i) { return bar_addr + 8u * (NS + i); };
    auto vfull = [&](int i) { return bar_addr + 8u * (2 * NS + i); };
    auto vempty = [&](int i) { return bar_addr + 8u * (3 * NS + i); };
    auto s_bar = [&](int g) { return bar_addr + 8u * (4 * NS + g); };         // S_g,j is there
    // (SEPARATE_P: all of it; else keys 0..63, and the others)
    auto s_high_bar = [&](int g) { return bar_addr + 8u * (4 * NS + 15 + g); };
    auto read_bar = [&](int g) { return bar_addr + 8u * (4 * NS + 2 + g); };  // and has been read
    auto o_bar = [&](int g) { return bar_addr + 8u * (4 * NS + 4 + g); };     // O_g has taken P_g,j
    // half of P_g,j is there
    auto p_bar = [&](int g, int hf) { return bar_addr + 8u * (4 * NS + 6 + 2 * hf + g); };
    auto drain_bar = [&](int g) { return bar_addr + 8u * (4 * NS + 10 + g); };
    const uint32_t q_bar = bar_addr + 8u * (4 * NS + 12);       // the Q tile is there
    const uint32_t z_bar = bar_addr + 8u * (4 * NS + 13);       // value rows past the end are zero
    const uint32_t start_bar = bar_addr + 8u * (4 * NS + 14);   // map 0 is half a tile ahead
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Sh::NBAR * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = p.num_kv_heads, Hq = p.num_heads, G = Hq / Hkv;
    const int TPB = Sh::BM / G;                   // chunk tokens per block
    // a cluster's blocks share out the keys of one query tile
    const int split = (int)cluster_size(), part = (int)cluster_rank();
    // the blocks of a unit take its query tiles, the last and longest first
    const int U = p.unit_tiles;
    const int unit = blockIdx.x / (split * U);
    const int ut = U - 1 - blockIdx.x / split % U;
    int h = unit % Hkv;

    if (warp == 0) {
        for (int i = lane; i < Sh::NBAR; i += 32) {
            const int k = i - 4 * NS;             // past the slots' barriers
            int count = 1;                        // a commit, or the producer
            if (k < 0)
                count = (i / NS) & 1 ? 2 : 1;     // empty: both maps' issuers
            else if ((k >= 2 && k < 4) || (k >= 6 && k < 10) || k == 14)
                count = 4;                        // read, p, start: one lane of each of 4 warps
            else if (k == 12 || k == 13)
                count = 8;                        // q, z: of every softmax warp
            mbar_init(bar_addr + 8u * i, count);
        }
        *abort_flag = 0;
        mbar_init_fence();
    }
    __syncwarp();

    // ---- the block's rows and key range (uniform over the block) ----------
    // no global memory is read before the preceding kernel (the plan) is done
    grid_dependency_wait();
    int s, rank = 0, tile = 0;
    if (p.plan) {
        if (!plan_block(p, unit, s, tile, h))
            return;
    } else {
        const int per_rank = p.num_seqs * Hkv;
        rank = unit / per_rank;
        s = (unit % per_rank) / Hkv;
    }
    const int L = __ldg(p.seq_lens + s);
    const int qs = __ldg(p.query_start + s);
    const int c = __ldg(p.query_start + s + 1) - qs;
    // the plan reports itself
    const bool reporter = !p.plan && rank == 0 && h == 0 && tid == 0 && ut == 0 && part == 0;
    if (L < 0 || L > p.max_blocks * kBlockSize) {
        if (reporter)
            record_error(p.err, PA_DEVERR_SEQLEN_RANGE);
        return;
    }
    if (c < 0 || c > L) {
        if (reporter)
            record_error(p.err, PA_DEVERR_QUERY_RANGE);
        return;
    }
    if (!p.plan) {
        const int nq = (c + U * TPB - 1) / (U * TPB);
        if (nq > p.q_ranks && reporter)
            record_error(p.err, PA_DEVERR_QUERY_RANGE);   // max_query_len too small
        if (rank >= nq)
            return;
        tile = nq - 1 - rank;                     // rank 0 = the last (longest) unit
    }
    const int t0 = (tile * U + ut) * TPB;
    if (t0 >= c)
        return;                                   // a unit's last tile may have no rows
    const int p_last = L - c + min(t0 + TPB, c) - 1;   // the tile's last row
    const int nt_all = p_last / Sh::BN + 1;       // key tiles, the same for the whole cluster
    // 2, 3, 4, 6, 8 or 16 of the cluster's blocks share them, two tiles or more each
    const int most = min(split, nt_all / 2);
    const int parts = most >= 16 ? 16 : most >= 8 ? 8 : most >= 6 ? 6 : max(1, min(most, 4));
    if (part >= parts)
        return;
    const int j0 = nt_all * part / parts;         // this block's first tile, and how many
    const int nt = nt_all * (part + 1) / parts - j0;
    // everything below counts keys, tiles and table entries from there
    const int Lk = L - j0 * Sh::BN;
    const int nblk = (Lk + kBlockSize - 1) / kBlockSize;
    // the last tile reaches past the sequence: its value rows there are zeroed
    const bool ragged = nt * Sh::BN > Lk;

    // What the block reads first is in flight over its last barrier: the block
    // table's first windows (producer), and the Q tile (softmax warps).  Q row
    // rr = (token t0 + rr / G, q head h*G + rr % G); rows past the chunk and the
    // rows 128 - TPB*G that do not fill a token are zero; thread lt takes 16-byte
    // chunk lt % CPR of every (256 / CPR)-th row.
    using Window = TableWindow<Sh::NB>;
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks + j0 * Sh::NB;
    constexpr int CPR = D / 8;                    // 16-byte chunks per row
    constexpr int RSTEP = 256 / CPR;
    constexpr int NPT = Sh::BM / RSTEP;
    const int lt = tid - 128;                     // softmax thread
    uint4 qv[NPT];
    int entry0 = 0, entry1 = 0;
    if (warp == 0) {
        entry0 = Window::fetch(table, nblk, 0);
        entry1 = Window::fetch(table, nblk, Window::WT);
        // K_0 at once
        Window w(p, table, h, nblk, entry0, entry1);
        const int row = w.row(0);
        if (lane == 0)
            mbar_arrive_expect_tx(kfull(0), (uint32_t)(min(Sh::NB, nblk) * Sh::HALVES * Sh::BOX));
        __syncwarp();
        if (lane < Sh::HALVES * Sh::NB && row >= 0)
            tma_load_2d(sbase + Sh::OFF_K + lane * Sh::BOX, &tmk, 64 * (lane / Sh::NB), row,
                        kfull(0));
    } else if (warp >= 4) {
        const T *qg = reinterpret_cast<const T *>(p.q);
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
            const int rr = lt / CPR + i * RSTEP;
            const int tok = rr / G, hg = rr % G;
            qv[i] = make_uint4(0, 0, 0, 0);
            if (rr < TPB * G && t0 + tok < c)
                qv[i] = __ldg(reinterpret_cast<const uint4 *>(
                    qg + ((size_t)(qs + t0 + tok) * Hq + h * G + hg) * D + (lt % CPR) * 8));
        }
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_addr(tmem_slot), Sh::TMEM_COLS);
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
        // ---------------- producer: K_j+1, V_j for every j ----------------
        // The whole warp works: lane 0 waits for the slot and arms its barrier,
        // lanes (hf, b) issue the tile's boxes in parallel.
        Window kw(p, table, h, nblk, entry0, entry1), vw = kw;
        auto load = [&](int j, int row, const CUtensorMap &tm, uint32_t slots, uint32_t full,
                        uint32_t empty) {
            bool ready = true;
            if (lane == 0)
                ready = !*abort_flag &&
                        (j < NS || mbar_wait_bounded(empty, (uint32_t)((j / NS - 1) & 1)));
            if (!__shfl_sync(FULL, ready, 0))
                return false;
            const int nv = min(Sh::NB, nblk - Sh::NB * j);
            if (lane == 0)
                mbar_arrive_expect_tx(full, (uint32_t)(nv * Sh::HALVES * Sh::BOX));
            __syncwarp();
            const int b = lane % Sh::NB, hf = lane / Sh::NB;
            if (hf < Sh::HALVES && row >= 0)
                tma_load_2d(slots + (j % NS) * Sh::SLOT_BYTES + (hf * Sh::NB + b) * Sh::BOX, &tm,
                            64 * hf, row, full);
            return true;
        };
        int nk = 1, nv = 0;                       // tiles issued: K_0 has been
        bool ok = true;
        for (int j = 0; ok && j < nt; ++j) {
            if (j + 1 < nt) {
                ok = load(j + 1, kw.row(j + 1), tmk, sbase + Sh::OFF_K, kfull((j + 1) % NS),
                          kempty((j + 1) % NS));
                nk += ok;
            }
            if (ok) {
                ok = load(j, vw.row(j), tmv, sbase + Sh::OFF_V, vfull(j % NS), vempty(j % NS));
                nv += ok;
            }
        }
        if (!ok && lane == 0 && !*abort_flag)
            give_up();
        // every issued copy lands before the block may exit
        if (lane < NS) {
            for (int j = max(0, nk - NS); j < nk; ++j)
                if (j % NS == lane && !mbar_wait_bounded(kfull(lane), (j / NS) & 1))
                    give_up();
            for (int j = max(0, nv - NS); j < nv; ++j)
                if (j % NS == lane && !mbar_wait_bounded(vfull(lane), (j / NS) & 1))
                    give_up();
        }
    } else if (warp <= 2) {
        // ---------------- MMA issuer of map g (the whole warp, one elected lane issues) ----
        const int g = warp - 1;
        constexpr uint32_t idO = tc::idesc_f16(kBf16, Sh::BM, D, false, true);
        // map 1's channels of the Q and K tiles start D/2 further: the next
        // 64-channel half, or 64 bytes into the row
        const uint32_t mo = g * (D == 128 ? Sh::BM * 128 : D);
        const uint64_t q_desc = tc::sdesc_sw128(sbase + mo, 16, 1024);
        const uint64_t k_desc = tc::sdesc_sw128(sbase + Sh::OFF_K + mo, 16, 1024);
        const uint64_t v_desc = tc::sdesc_sw128(sbase + Sh::OFF_V, Sh::NB * Sh::BOX, 1024);
        const uint32_t ts = tmem + g * Sh::MAP_COLS, tp = ts + Sh::COL_P, to = ts + Sh::COL_O;
        static_assert(Sh::BM * 128 == Sh::NB * Sh::BOX, "Q and K halves 16 KB apart");
        // a slot's wait costs 100 to 250 cycles even when its copy has long
        // landed, so it comes before the wait for the softmax or the last P.V
        auto k_ready = [&](int j) { return mbar_wait_warp(kfull(j % NS), (j / NS) & 1); };
        auto v_ready = [&](int j) { return mbar_wait_warp(vfull(j % NS), (j / NS) & 1); };
        // a slot is free once both maps have read tile j; said of slots that a later
        // tile takes
        auto release = [&](uint32_t bar, int j) {
            if (j + NS < nt)
                tc::commit_warp(bar);
        };
        // S of tile j: all of it, or (P over S) half hf of its keys
        auto issue_s = [&](int j, int hf) {
            constexpr int N = Sh::SEPARATE_P ? Sh::BN : Sh::BN / 2;
            constexpr uint32_t idS = tc::idesc_f16(kBf16, Sh::BM, N, false, false);
            const int sl = j % NS;
            tc::fence_after_sync();
            const uint64_t kd =
                k_desc + (uint64_t)((sl * Sh::SLOT_BYTES + hf * N * 128) >> 4);
#pragma unroll
            for (int k = 0; k < D / 32; ++k)      // 32 bytes along the 128-byte row a step
                tc::mma_ss_warp(ts + hf * N, q_desc + 2 * k, kd + 2 * k, idS, k > 0);
            tc::commit_warp(hf ? s_high_bar(g) : s_bar(g));
            if (Sh::SEPARATE_P || hf)
                release(kempty(sl), j);
        };
        // O_g += P_g,j . V_j, each half of the keys once the softmax has written
        // its P
        auto issue_pv = [&](int j) -> bool {
            const int sl = j % NS;
            const uint64_t vd = v_desc + (uint64_t)((sl * Sh::SLOT_BYTES) >> 4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                if (!mbar_wait_warp(p_bar(g, hf), j & 1))
                    return false;
                tc::fence_after_sync();
#pragma unroll
                for (int kk = 4 * hf; kk < 4 * hf + 4; ++kk)
                    // A = P: keys 16kk.. = 8 packed columns; B = V block kk (MN-major:
                    // 64-channel groups NB boxes apart, 8-key groups 1 KB apart)
                    tc::mma_ts_warp(to, tp + 8 * kk, vd + (uint64_t)((kk * Sh::BOX) >> 4), idO,
                                    (j > 0 || kk > 0) ? 1u : 0u);
            }
            tc::commit_warp(o_bar(g));
            release(vempty(sl), j);
            return true;
        };
        // map 1 starts half a tile behind: the maps' softmaxes then alternate on the
        // sub-cores and their MMAs on the tensor core, for a while (1146 us against 1156
        // on two 2048-token chunks at 16K, 195 against 199 on 8 x 512 tokens)
        bool ok = k_ready(0) && mbar_wait_warp(q_bar, 0) &&
                  (g == 0 || mbar_wait_warp(start_bar, 0));
        if (ok)
            issue_s(0, 0);
        if (ok && !Sh::SEPARATE_P)
            issue_s(0, 1);
        for (int j = 0; ok && j < nt; ++j) {
            const bool more = j + 1 < nt;
            // V_j is waited for before S_g,j+1 goes out at head_dim 64, where that has
            // time (2 x 2048 tokens at 16K: 982 us against 999), after it at 128
            ok = (!Sh::SEPARATE_P ||
                  (v_ready(j) && (!ragged || more || mbar_wait_warp(z_bar, 0)))) &&
                 (!more || k_ready(j + 1));
            // S_g,j+1, or its first half, only needs the softmax to have read S_g,j's
            if (ok && more && (ok = mbar_wait_warp(read_bar(g), j & 1)))
                issue_s(j + 1, 0);
            ok = ok &&
                 (Sh::SEPARATE_P ||
                  (v_ready(j) && (!ragged || more || mbar_wait_warp(z_bar, 0)))) &&
                 issue_pv(j);
            // the second half goes where P_g,j was
            if (!Sh::SEPARATE_P && ok && more && (ok = mbar_wait_warp(o_bar(g), j & 1)))
                issue_s(j + 1, 1);
        }
        if (!ok && lane == 0)
            give_up();
        // no MMA may still run when TMEM is freed
        tc::commit_warp(drain_bar(g));
        if (!mbar_wait_warp(drain_bar(g), 0) && lane == 0)
            give_up();
    } else if (warp == 3) {
        // while the block works: warm L2 with the query rows of the block one
        // wave later (its pair and kv head from the work order)
        int s2, tile2, h2;
        const int b2 = blockIdx.x + p.wave;
        if (p.plan && plan_block(p, b2 / U, s2, tile2, h2)) {
            const int qs2 = __ldg(p.query_start + s2);
            const int t02 = (tile2 * U + U - 1 - b2 % U) * TPB;
            const int ntok = min(TPB, __ldg(p.query_start + s2 + 1) - qs2 - t02);
            const int lines = G * D * 2 / 128;      // 128-byte lines of a token's G heads
            const T *qg = reinterpret_cast<const T *>(p.q);
            for (int i = lane; i < ntok * lines; i += 32)
                prefetch_l2(qg + ((size_t)(qs2 + t02 + i / lines) * Hq + h2 * G) * D +
                            (i % lines) * 64);
        }
    } else if (warp >= 4) {
        // ---------------- Q tile -> shared memory ----------------
        // K-major with the 128-byte swizzle
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
            const int rr = lt / CPR + i * RSTEP, ch = lt % CPR;
            *reinterpret_cast<uint4 *>(smem + (ch >> 3) * (Sh::BM * 128) + rr * 128 +
                                       (((ch & 7) ^ (rr & 7)) << 4)) = qv[i];
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(q_bar);

        // ---------------- softmax: one thread per row of its map ----------
        const int grp = (warp - 4) >> 2;
        const int q4 = warp & 3;                   // TMEM lane quarter of this warp
        const int rr = q4 * 32 + lane;             // row
        const uint32_t lanes = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t tg = lanes + grp * Sh::MAP_COLS;
        const int tok = rr / G, hg = rr % G;
        const bool row_valid = rr < TPB * G && t0 + tok < c;
        const int pos = (row_valid ? L - c + t0 + tok : L - 1) - j0 * Sh::BN;
        const float sl2 = p.scale_log2;
        const float lam = __ldg(p.lambda + h * G + hg);
        auto arrive = [&](uint32_t bar) {          // once a warp, after its lanes' work
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
        };
        float m = 0.f, l = 0.f;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            if (!mbar_wait_warp(s_bar(grp), j & 1)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const int k0 = j * Sh::BN;
            const int vis = pos - k0;              // keys [0, vis] of the tile are visible
            // the 128 scores of the row, both halves held in registers; the first
            // half's maximum is taken while the second half is on its way
            uint32_t v[2][64];
            // tiles left of the diagonal (the common case) need no mask
            const bool full = __all_sync(FULL, vis >= Sh::BN - 1);
            auto mask = [&](int from, int to) {
                if (!full) {
#pragma unroll
                    for (int e = 0; e < Sh::BN; ++e)
                        if (e >= from && e < to && e > vis)
                            v[e >> 6][e & 63] = __float_as_uint(-INFINITY);
                }
            };
            auto x = [&](int i) { return __uint_as_float(v[i >> 6][i & 63]); };
            float mx[8];                         // trees, three operands per instruction
            __syncwarp();                        // tcgen05.ld is warp-collective
            tc::tmem_ld64(tg, v[0]);
            if constexpr (Sh::SEPARATE_P)
                tc::tmem_ld64(tg + 64, v[1]);
            tc::fence_before_sync();
            arrive(read_bar(grp));               // S_g,j+1 (its first half) may go in
            mask(0, Sh::SEPARATE_P ? Sh::BN : 64);
#pragma unroll
            for (int a = 0; a < 8; ++a) {
                float t = fmax3(x(a), x(a + 8), x(a + 16));
                t = fmax3(t, x(a + 24), x(a + 32));
                t = fmax3(t, x(a + 40), x(a + 48));
                mx[a] = fmaxf(t, x(a + 56));
            }
            if constexpr (!Sh::SEPARATE_P) {
                if (!mbar_wait_warp(s_high_bar(grp), j & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                __syncwarp();
                tc::tmem_ld64(tg + 64, v[1]);
                mask(64, Sh::BN);
            }
#pragma unroll
            for (int a = 0; a < 8; ++a) {
                float t = fmax3(mx[a], x(a + 64), x(a + 72));
                t = fmax3(t, x(a + 80), x(a + 88));
                t = fmax3(t, x(a + 96), x(a + 104));
                mx[a] = fmax3(t, x(a + 112), x(a + 120));
            }
            float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                             fmaxf(mx[6], mx[7]));
            mt *= sl2;                           // scale > 0: max commutes with it
            // running maximum, raised lazily: only when the tile's maximum
            // exceeds it by more than 8 (P stays below 2^8 otherwise)
            bool grow = false;
            float alpha = 1.f;
            if (j == 0) {
                m = fmaxf(mt, -3e38f);           // finite also if every score is -inf
            } else if (mt > m + 8.f) {
                grow = true;
                alpha = ex2_approx(m - mt);
                m = mt;
            }
            // P = 2^(scale*s - m) packed to the operand type; scale-and-subtract
            // and the row sum run two values per instruction
            const uint64_t sl2x2 = f2_pack(sl2, sl2), nmx2 = f2_pack(-m, -m);
            uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t pw[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    float y0, y1;
                    const uint64_t x2 = f2_pack(__uint_as_float(v[hf][e]),
                                                __uint_as_float(v[hf][e + 1]));
                    f2_unpack(f2_fma(x2, sl2x2, nmx2), y0, y1);
                    const float p0 = ex2_approx(y0);
                    const float p1 = ex2_approx(y1);
                    sum2[(e >> 1) & 3] = f2_add(sum2[(e >> 1) & 3], f2_pack(p0, p1));
                    pw[e / 2] = Mma<T>::pack(p0, p1);
                }
                if (Sh::SEPARATE_P && hf == 0) {
                    // P_g,j overwrites P_g,j-1, and O may be rescaled below: both
                    // wait for P_g,j-1 . V_j-1 (with P over S, S_g,j came after it)
                    if (j > 0 && !mbar_wait_warp(o_bar(grp), (j - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                }
                __syncwarp();
                tc::tmem_st32(tg + Sh::COL_P + 32 * hf, pw);
                if (hf == 0) {
                    // value rows of keys >= L are zeroed (0 * NaN is NaN in the
                    // MMA), by both maps' threads; both issuers wait for all of them
                    if (ragged && j == nt - 1) {
                        const int sl = j % NS;
                        if (!mbar_wait_warp(vfull(sl), (j / NS) & 1)) {
                            ok = false;
                            break;
                        }
                        const int first = Lk - k0;
                        const int n16 = (Sh::BN - first) * Sh::HALVES * 8;
                        unsigned char *vb = smem + Sh::OFF_V + sl * Sh::SLOT_BYTES;
                        for (int idx = lt; idx < n16; idx += 256) {
                            const int row = first + idx / (Sh::HALVES * 8);
                            const int rem = idx % (Sh::HALVES * 8);
                            unsigned char *at = vb +
                                                ((rem >> 3) * Sh::NB + (row >> 4)) * Sh::BOX +
                                                (row & 15) * 128 + (rem & 7) * 16;
                            *reinterpret_cast<uint4 *>(at) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_shared();
                        arrive(z_bar);
                    }
                    // O rescale: P_g,j-1 . V_j-1 has completed
                    if (__any_sync(FULL, grow)) {
#pragma unroll
                        for (int cc = 0; cc < D; cc += 32) {
                            uint32_t o[32];
                            tc::tmem_ld32(tg + Sh::COL_O + cc, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tc::tmem_st32(tg + Sh::COL_O + cc, o);
                        }
                    }
                }
                tc::fence_before_sync();
                arrive(p_bar(grp, hf));
                if (j == 0 && hf == 0 && grp == 0)
                    arrive(start_bar);
            }
            if (!ok)
                break;
            float sum[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float a, b;
                f2_unpack(sum2[q], a, b);
                sum[q] = a + b;
            }
            l = fmaf(l, alpha, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        }
        if (parts > 1) {
            // ---------------- this block's keys' share, for join_split ----------------
            if (ok && !mbar_wait_warp(o_bar(grp), (nt - 1) & 1))
                ok = false;
            if (!ok)
                give_up();
            float *xs = reinterpret_cast<float *>(smem + Sh::OFF_X);  // [sum, maximum][2][128]
            xs[grp * Sh::BM + rr] = l;
            xs[(2 + grp) * Sh::BM + rr] = m;
            // past this barrier both maps' MMAs are done with the K and V tiles
            tc::fence_before_sync();
            softmax_warps_sync();
            tc::fence_after_sync();
            if (!__any_sync(FULL, *abort_flag != 0)) {
                float4 *to = reinterpret_cast<float4 *>(smem + Sh::OFF_K) +
                             (size_t)(grp * Sh::BM + rr) * (D / 4);
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tc::tmem_ld32(tg + Sh::COL_O + cc, o);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        to[((cc + e) / 4) ^ (rr & 7)] =
                            make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                        __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                }
            }
        } else {
            // ---------------- the difference, its norm, the output ----------------
            // This thread's half of the channels; the norm's weights are in flight
            // over the last P.V.
            constexpr int HC = D / 2, CH = HC / 8;    // channels, 16-byte chunks
            uint4 wv[CH];
            const bool normed = p.norm_w != nullptr;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                wv[i] = normed ? __ldg(reinterpret_cast<const uint4 *>(
                                           static_cast<const T *>(p.norm_w) + grp * HC) + i)
                               : make_uint4(0, 0, 0, 0);
            if (ok && !mbar_wait_warp(o_bar(grp), (nt - 1) & 1))
                ok = false;
            // Row sums and the halves' sums of squares go through shared memory.
            // Every softmax thread takes part in both barriers, also after a wait that
            // gave up; past the first, both maps' last P.V are known to be done.
            float *xl = reinterpret_cast<float *>(smem + Sh::OFF_X);      // [2][128]
            float *xq = xl + 2 * Sh::BM;                                  // [2][128]
            if (!ok)
                give_up();
            xl[grp * Sh::BM + rr] = l;
            tc::fence_before_sync();
            softmax_warps_sync();
            tc::fence_after_sync();
            ok = !__any_sync(FULL, *abort_flag != 0);
            const float i0 = 1.f / xl[rr];
            const float i1 = -lam / xl[Sh::BM + rr];
            const uint32_t half = lanes + Sh::COL_O + grp * HC;
            float y[HC], ss = 0.f;
            if (ok) {
#pragma unroll
                for (int cc = 0; cc < HC; cc += 32) {
                    uint32_t a[32], b[32];
                    __syncwarp();
                    tc::tmem_ld32(half + cc, a);
                    tc::tmem_ld32(half + Sh::MAP_COLS + cc, b);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        y[cc + e] = fmaf(__uint_as_float(b[e]), i1, __uint_as_float(a[e]) * i0);
                        ss = fmaf(y[cc + e], y[cc + e], ss);
                    }
                }
            }
            xq[grp * Sh::BM + rr] = ss;
            softmax_warps_sync();
            if (ok) {
                float k = p.out_scale;
                if (normed)
                    k *= rsqrtf((xq[rr] + xq[Sh::BM + rr]) * (1.f / D) + p.norm_eps);
                // Through the warp's part of the Q tile's shared memory (no MMA reads
                // Q any more), so that a warp's stores are whole 128-byte lines: a
                // row to a thread, they touched 32 lines an instruction.
                uint4 *st = reinterpret_cast<uint4 *>(smem) + (warp - 4) * 32 * CH;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    float f[8];
                    const uint32_t w32[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 x = normed ? Elem<T>::to_f2(w32[e]) : make_float2(1.f, 1.f);
                        f[2 * e] = y[8 * i + 2 * e] * (k * x.x);
                        f[2 * e + 1] = y[8 * i + 2 * e + 1] * (k * x.y);
                    }
                    st[lane * CH + (i ^ (lane % CH))] =
                        make_uint4(Mma<T>::pack(f[0], f[1]), Mma<T>::pack(f[2], f[3]),
                                   Mma<T>::pack(f[4], f[5]), Mma<T>::pack(f[6], f[7]));
                }
                __syncwarp();
                const long long mine =
                    row_valid ? ((long long)(qs + t0 + tok) * Hq + h * G + hg) * D + grp * HC : -1;
                T *out = reinterpret_cast<T *>(p.out);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int row = i * (32 / CH) + lane / CH, ch = lane % CH;
                    const long long at = __shfl_sync(FULL, mine, row);
                    if (at >= 0)
                        *reinterpret_cast<uint4 *>(out + at + 8 * ch) =
                            st[row * CH + (ch ^ (row % CH))];
                }
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, Sh::TMEM_COLS);
    }
    if (parts > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp >= 4) {
            const uint32_t aborts = smem_addr(const_cast<int *>(abort_flag));
            const int rows = min(TPB, c - t0) * G;
            const size_t token = (size_t)(qs + t0);
            auto join = [&](auto se) {
                join_split<T, D, decltype(se)::value>(p, sbase, aborts, part, lt, rows, G, h,
                                                      token);
            };
            switch (parts) {
            case 16: join(std::integral_constant<int, 16>{}); break;
            case 8: join(std::integral_constant<int, 8>{}); break;
            case 6: join(std::integral_constant<int, 6>{}); break;
            case 4: join(std::integral_constant<int, 4>{}); break;
            case 3: join(std::integral_constant<int, 3>{}); break;
            default: join(std::integral_constant<int, 2>{}); break;
            }
        }
        // no block ends while another reads its shared memory
        __syncwarp();
        cluster_arrive_relaxed();
        cluster_wait();
    }
}

template <typename T, int D>
void entry(PrefillKernel *k)
{
    k->fn = reinterpret_cast<const void *>(&diff_prefill_kernel_t<T, D>);
    k->threads = DiffShape<D>::THREADS;
    k->smem = DiffShape<D>::SMEM;
}

}  // namespace

bool diff_prefill_kernel(int dtype, int head_dim, PrefillKernel *k)
{
    // the work order is the plain prefill's
    if (!prefill_kernel(dtype, head_dim, k))
        return false;
    const bool bf = dtype == PA_DTYPE_BF16;
    if (head_dim == 64)
        bf ? entry<__nv_bfloat16, 64>(k) : entry<__half, 64>(k);
    else
        bf ? entry<__nv_bfloat16, 128>(k) : entry<__half, 128>(k);
    return true;
}

}  // namespace pa
