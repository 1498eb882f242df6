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
// tokens of a (sequence, kv head), four a lane a stride of 32 apart.  The batch-128
// decode step, 32/8 heads: 19.2 MB in 8.4 us of the 88.1 that decode and accounting take in
// a graph of one batch (the plain decode 77.7, leaving the scores 2; 92.5 and 78.2 where three
// batches take turns and L2 keeps nothing): two or three runs a warp, each a chain of length,
// statistics and scores.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kMassFinishThreads, 4)
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
            const float2 *x = reinterpret_cast<const float2 *>(p.scores + (run * T + t0) * cols);
            const float2 *stat = p.stat + (size_t)s * p.num_heads + h * G;
            float *mass = p.mass + run * T + t0;
            // every load of four heads in flight at once, and the old masses with the first
            // (the newest token has none from before)
            const int step = 16 * cols;           // 32 tokens, in pairs of scores
            float old[4], sum[4];
            bool on[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                on[k] = t0 + 32 * k < L;
                old[k] = t0 + 32 * k < L - 1 && p.decay != 0.f ? __ldcg(mass + 32 * k) : 0.f;
                sum[k] = 0.f;
            }
            for (int g = 0; g < cols; g += 4) {
                // heads past the group: a reciprocal of 0
                float2 st[4], y[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st[i] = g + i < G ? __ldcg(stat + g + i) : make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k][i] = on[k] && g + 2 * i < cols ? __ldcg(x + k * step + g / 2 + i)
                                                            : make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // (the odd group's last score of a pair is that of a query of zeros: finite)
                    const float2 a = st[2 * i], b = st[2 * i + 1];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sum[k] = fmaf(ex2_approx(y[k][i].x - a.x), a.y,
                                      fmaf(ex2_approx(y[k][i].y - b.x), b.y, sum[k]));
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (on[k])
                    mass[32 * k] = fmaf(old[k], p.decay, sum[k]);
        }
    }
}

// ---------------------------------------------------------------------------
// A chunk of queries, on the fifth-generation tensor cores.  A unit of work is
// 2 x 128 (token, head) rows of a (sequence, kv head); they stay in
// place while the sequence's keys stream past in 128-key tiles (TMA, a ring of
// slots).  Pass 1 (SUMS false) takes S = Q.K^T, a thread a query row, and leaves
// each row's maximum and sum; pass 2 takes S^T = K.Q^T, a thread a key, so that
// the sum over the queries is a sum over the thread's own columns, with the
// row's statistics read from shared memory as a broadcast.
//
// Shared memory's bandwidth is what a 128 x 128 product of two operands there
// uses up (128 bytes a cycle, before the copies): pass 1 keeps its query rows in
// tensor memory, beside three buffers of scores that its query tiles take in
// turn, and pass 2 multiplies a key tile by both query tiles at once (128 x 256),
// two buffers.  Four sets of four warps take the exponentials, two of each query
// tile: in pass 1 a set takes 64 keys of every key tile, so that a buffer is
// free again as soon as it has been loaded (with 128 keys of every other one in
// two steps, half of a set's time later, the products waited for the three
// buffers); in pass 2, where a buffer's two tiles' time is longer, it takes the 128
// rows of every other key tile, so that a key's sum over a query tile is one
// thread's.
//
// The key tiles of all units form one list, ordered by sequence, kv head and
// row block; each block of the persistent grid takes an equal share of it.  A
// unit cut by a share's border has a piece in each of several blocks; piece
// statistics go to slot (unit + block), which no two pieces have in common
// since both grow along the list.  Pass 2 folds a unit's pieces when it loads its
// rows, and reads each piece's keys from the last tile back: those are the ones
// that pass 1 left in L2.
//
// 64 rows x 4 heads over 8 sequences of 16K tokens, 8 kv heads x 128: 127 us in a graph,
// 63 a pass, each 268 MB of keys and 68.7 GFLOP (4.2 TB/s and 1.08 PFLOP/s over the
// two).  No one unit is full: the tensor pipe is active 42 % of the time,
// the exponentials' 43 %, issue slots 53 %; 13 us a pass are its start and end.  Without
// exponentials pass 1 takes 57 us, with its keys in L2 as well 55: what is left is the
// products' hand-overs, 0.78 us a tile of 128 keys against 0.66 at the library's rate.
// ---------------------------------------------------------------------------
template <int D, bool SUMS>
struct MassShape {
    static constexpr int BM = kMassRows, NG = kMassTiles, BN = kMassKeys;
    static constexpr int NB = BN / kBlockSize;
    static constexpr int HALVES = D / 64;
    static constexpr int BOX = 2048;                      // 16 rows x 128 B
    static constexpr int Q_BYTES = SUMS ? NG * BM * D * 2 : 0;   // [half][256 rows][128 B]
    static constexpr int SLOT_BYTES = BN * D * 2;         // [half][8 blocks][16 rows][128 B]
    static constexpr int NSLOT = D == 64 ? 8 : SUMS ? 4 : 6;
    static constexpr int OFF_SLOT = Q_BYTES;
    static constexpr int OFF_LSE = OFF_SLOT + NSLOT * SLOT_BYTES;
    static constexpr int OFF_PART = OFF_LSE + 2 * NG * BM * 4;   // [buffer][turn & 1][key]
    // full[NSLOT] empty[NSLOT] s[4] read[3] q[2] free[2] group[2] sum[4] drain, then TMEM base
    // and abort flag
    static constexpr int NBAR = 2 * NSLOT + 18;
    static constexpr int OFF_BAR = OFF_PART + (SUMS ? 4 * BN * 4 : 0);
    static constexpr int SMEM = 1024 + OFF_BAR + NBAR * 8 + 8;
    static constexpr int THREADS = 64 + NG * 256;
    // tensor memory: score buffers of 128 (pass 1) or 256 columns, pass 1's query rows
    static constexpr uint32_t COL_Q = 384;
    static_assert(SMEM <= 227 * 1024, "one block per SM");
};

// A sequence's chunk: its first row of q, rows, length and the end of its row blocks that this
// launch takes (0: nothing to do; up to block0: nothing in this launch).
struct MassSeq {
    int L, c, qs, blocks;
};

__device__ __forceinline__ MassSeq mass_seq(const PrefillMassParams &p, int s, int TPB, bool report)
{
    MassSeq x;
    x.L = __ldg(p.seq_lens + s);
    x.qs = __ldg(p.query_start + s);
    x.c = __ldg(p.query_start + s + 1) - x.qs;
    x.blocks = 0;
    if (x.L < 0 || x.L > p.max_blocks * kBlockSize) {
        if (report)
            record_error(p.err, PA_DEVERR_SEQLEN_RANGE);
    } else if (x.c < 0 || x.c > x.L || x.qs < 0 || x.c > p.num_queries - x.qs ||
               (x.c + TPB - 1) / TPB > p.all_blocks) {
        if (report)
            record_error(p.err, PA_DEVERR_QUERY_RANGE);
    } else {
        x.blocks = min((x.c + TPB - 1) / TPB, p.block0 + p.row_blocks);
    }
    return x;
}

// Key tiles that row block b sees: up to its last row.
__device__ __forceinline__ int mass_tiles(const MassSeq &x, int b, int TPB)
{
    return (x.L - x.c + min((b + 1) * TPB, x.c) - 1) / kMassKeys + 1;
}

// Those of the launch's row blocks.
__device__ __forceinline__ int mass_tiles(const PrefillMassParams &p, const MassSeq &x, int TPB)
{
    int n = 0;
    for (int b = p.block0; b < x.blocks; ++b)
        n += mass_tiles(x, b, TPB);
    return n;
}

// One thread block's way along the list of key tiles.
struct MassWalker {
    MassSeq x;
    int s, h, b;                   // sequence, kv head, row block
    int first, nt;                 // the unit's first tile in the list, its tiles
    int tb, te;                    // this piece's tiles of the unit
    int end;                       // of the share
    bool valid;

    __device__ __forceinline__ void piece(int TPB, int from)
    {
        nt = mass_tiles(x, b, TPB);
        tb = from - first;
        te = min(nt, end - first);
    }

    // Start at place `at` of the list; sequence s0 begins at `from`.
    __device__ __forceinline__ void init(const PrefillMassParams &p, int TPB, int s0, int from,
                                         int at, int end_)
    {
        end = end_;
        valid = at < end;
        if (!valid)
            return;
        s = s0;
        x = mass_seq(p, s, TPB, false);
        const int per = mass_tiles(p, x, TPB);
        h = (at - from) / per;
        first = from + h * per;
        b = p.block0;
        while (first + mass_tiles(x, b, TPB) <= at)
            first += mass_tiles(x, b++, TPB);
        piece(TPB, at);
    }

    __device__ __forceinline__ void next(const PrefillMassParams &p, int TPB)
    {
        first += nt;
        valid = first < end;
        if (!valid)
            return;
        if (++b == x.blocks) {
            b = p.block0;
            if (++h == p.num_kv_heads) {
                h = 0;
                do
                    x = mass_seq(p, ++s, TPB, false);
                while (x.blocks <= p.block0);
            }
        }
        piece(TPB, first);
    }
};

template <typename T, int D, bool SUMS>
__global__ void __launch_bounds__(MassShape<D, SUMS>::THREADS)
prefill_mass_kernel(const PrefillMassParams p, const __grid_constant__ CUtensorMap tmk)
{
    using Sh = MassShape<D, SUMS>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int NS = Sh::NSLOT, NTH = Sh::THREADS, ROWS = Sh::NG * Sh::BM;
    extern __shared__ unsigned char smem_raw[];
    __shared__ int scan[NTH / 32], start_seq, start_at;
    const uint32_t raw_addr = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_addr(smem), slot_addr = sbase + Sh::OFF_SLOT;
    float *lse = reinterpret_cast<float *>(smem + Sh::OFF_LSE);      // [unit & 1] minus log sums
    float *part = reinterpret_cast<float *>(smem + Sh::OFF_PART);    // the first query tile's sums
    const uint32_t bar_addr = sbase + Sh::OFF_BAR;
    auto full_bar = [&](int s) { return bar_addr + 8u * s; };
    auto empty_bar = [&](int s) { return bar_addr + 8u * (NS + s); };
    // scores are there (pass 1: for a query tile's every other turn; pass 2: in a buffer); a
    // buffer has been read; query rows are there; a piece's products have ended
    auto s_bar = [&](int i) { return bar_addr + 8u * (2 * NS + i); };
    auto read_bar = [&](int b) { return bar_addr + 8u * (2 * NS + 4 + b); };
    auto q_bar = [&](int g) { return bar_addr + 8u * (2 * NS + 7 + g); };
    auto free_bar = [&](int g) { return bar_addr + 8u * (2 * NS + 9 + g); };
    auto group_bar = [&](int g) { return bar_addr + 8u * (2 * NS + 11 + g); };
    auto sum_bar = [&](int i) { return bar_addr + 8u * (2 * NS + 13 + i); };
    const uint32_t drain_bar = bar_addr + 8u * (2 * NS + 17);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Sh::OFF_BAR + Sh::NBAR * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = p.num_kv_heads, Hq = p.num_heads, G = Hq / Hkv;
    const int TPG = Sh::BM / G, TPB = Sh::NG * TPG;       // chunk tokens of a tile, of a unit
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_bar(i), 1);
            mbar_init(sum_bar(i), 128);
        }
        for (int i = 0; i < 3; ++i)
            mbar_init(read_bar(i), 256);
        for (int g = 0; g < Sh::NG; ++g) {
            mbar_init(q_bar(g), SUMS ? 512 : 256);
            mbar_init(free_bar(g), 1);
            mbar_init(group_bar(g), 256);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) {                              // (no two of these blocks fit on an SM)
        tc::tmem_alloc(smem_addr(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    // Pass 2 may be scheduled once every block of pass 1 is past the wait for what came before
    // both: it then reads the caller's arrays at once, and waits for pass 1 where it reads
    // statistics.
    if (!SUMS) {
        grid_dependency_wait();
        grid_dependents_launch();
    }

    // ---- the block's share: the list's length, then the sequence its share starts in ----
    auto tiles_of = [&](int s, bool report) {
        const MassSeq x = mass_seq(p, s, TPB, report);
        return Hkv * mass_tiles(p, x, TPB);
    };
    int carry = 0, mine = 0, before = 0;          // of this thread's last sequence
    auto scan_from = [&](int s0, bool report) {
        const int s = s0 + tid;
        mine = s < p.num_seqs ? tiles_of(s, report && !SUMS && blockIdx.x == 0) : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, incl, o);
            if (lane >= o)
                incl += y;
        }
        __syncthreads();                          // scan has been read
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        before = carry + incl - mine;
#pragma unroll
        for (int w = 0; w < NTH / 32; ++w) {
            before += w < warp ? scan[w] : 0;
            carry += scan[w];
        }
    };
    for (int s0 = 0; s0 < p.num_seqs; s0 += NTH)
        scan_from(s0, true);
    const int total = carry;
    const int R = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const long long share = (long long)blockIdx.x * R;
    if (share < total) {
        const int at = (int)share;
        auto found = [&](int s0) {
            if (mine > 0 && before <= at && at < before + mine) {
                start_seq = s0 + tid;
                start_at = before;
            }
        };
        if (p.num_seqs <= NTH) {
            found(0);
        } else {
            carry = 0;
            for (int s0 = 0; s0 < p.num_seqs && carry <= at; s0 += NTH) {
                scan_from(s0, false);
                found(s0);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    MassWalker w;
    w.init(p, TPB, start_seq, start_at, (int)min(share, (long long)total),
           (int)min((long long)total, share + R));
    auto give_up = [&]() {
        *abort_flag = 1;
        record_error(p.err, PA_DEVERR_TIMEOUT);
    };
    // query tiles of the piece's unit that have rows
    auto groups = [&]() { return w.x.c - w.b * TPB > TPG ? 2 : 1; };
    // the piece's i-th key tile
    auto tile = [&](int i) { return SUMS ? w.te - 1 - i : w.tb + i; };

    if (warp == 0) {
        // ---------------- producer: key tiles into the ring ----------------
        // lane l holds the pool row of block NB * win + l of a window of WT tiles, and the next
        // window's table entries are in flight; lane 0 waits for the slot, lanes (half,
        // block) issue the boxes
        constexpr int NB = Sh::NB, WT = 32 / NB;
        int it = 0, last = -1;                    // last: the last tile in this lane's slot
        bool ok = true;
        for (; ok && w.valid; w.next(p, TPB)) {
            const int nblk = (w.x.L + kBlockSize - 1) / kBlockSize;
            const int32_t *table = p.block_tables + (size_t)w.s * p.max_blocks;
            auto fetch = [&](int w0) {
                const int lb = NB * w0 + lane;
                return w0 >= 0 && lb < nblk ? __ldg(table + lb) : 0;
            };
            auto to_row = [&](int w0, int phys) {
                if (NB * w0 + lane >= nblk)
                    return -1;
                if ((unsigned)phys >= (unsigned)p.num_blocks) {
                    record_error(p.err, PA_DEVERR_TABLE_RANGE);
                    phys = 0;
                }
                return (phys * Hkv + w.h) * kBlockSize;
            };
            const int step = SUMS ? -WT : WT;
            int win = tile(0) / WT * WT;
            int cur = to_row(win, fetch(win));
            int nxt = fetch(win + step);
            for (int i = 0; i < w.te - w.tb; ++i, ++it) {
                const int j = tile(i), sl = it % NS;
                if (j / WT * WT != win) {
                    win += step;
                    cur = to_row(win, nxt);
                    nxt = fetch(win + step);
                }
                // (the bounded waits of pass 2 begin once pass 1, which they wait for too, has ended)
                if (SUMS && it == NS)
                    grid_dependency_wait();
                bool ready = true;
                if (lane == 0)
                    ready = !*abort_flag &&
                            (it < NS || mbar_wait_bounded(empty_bar(sl), ((it / NS) - 1) & 1));
                if (!__shfl_sync(FULL, ready, 0)) {
                    if (lane == 0 && !*abort_flag)
                        give_up();
                    ok = false;
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
                    last = it;
            }
        }
        // every issued copy lands before the block may exit
        if (lane < NS && last >= 0 && !mbar_wait_bounded(full_bar(lane), (last / NS) & 1))
            give_up();
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t id128 = tc::idesc_f16(kBf16, 128, 128, false, false);
        constexpr uint32_t id256 = tc::idesc_f16(kBf16, 128, 256, false, false);
        const uint64_t q_desc = tc::sdesc_sw128(sbase, 16, 1024);
        const uint64_t k_desc = tc::sdesc_sw128(slot_addr, 16, 1024);
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(FULL, mbar_wait_bounded(bar, parity));
        };
        bool ok = true;
        int it = 0;                               // key tiles so far
        int rows[Sh::NG] = {0, 0};                // units so far of each query tile
        int turn[Sh::NG] = {0, 0};                // key tiles so far of each query tile
        uint32_t used = 0, odd = 0;               // of each score buffer: used yet, parity
        if (SUMS)                                 // the rows come after it
            grid_dependency_wait();
        for (; ok && w.valid; w.next(p, TPB)) {
            const int ng = groups();
            for (int i = 0; ok && i < w.te - w.tb; ++i, ++it) {
                const int sl = it % NS;
                const uint64_t kd = k_desc + (uint64_t)((sl * Sh::SLOT_BYTES) >> 4);
                if (__any_sync(FULL, *abort_flag != 0) ||
                    !wait_all(full_bar(sl), (it / NS) & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int g = 0; g < (SUMS ? 1 : Sh::NG); ++g) {
                    if (g >= ng || !ok)
                        continue;
                    const int buf = SUMS ? it & 1 : ng == 2 ? (2 * i + g) % 3 : i & 1;
                    if (i == 0)
                        ok = wait_all(q_bar(g), rows[g]++ & 1);
                    // The buffer's last scores have been read; and with them, three tiles (one
                    // query tile: two) before, what the warps were given two turns before:
                    // they never have more ahead of them than two barriers tell apart.
                    if (ok && (used >> buf & 1))
                        ok = wait_all(read_bar(buf), ~odd >> buf & 1);
                    used |= 1u << buf;
                    odd ^= 1u << buf;
                    if (!ok)
                        continue;
                    tc::fence_after_sync();
                    // a K step: 32 bytes along the 128-byte row; the next 64 channels are a half
                    // further
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t ko =
                            (uint64_t)(((k & 3) * 32 + (k >> 2) * (128 * 128)) >> 4);
                        if (SUMS)
                            tc::mma_ss_warp(
                                tmem + 256 * buf, kd + ko,
                                q_desc + (uint64_t)(((k & 3) * 32 + (k >> 2) * (256 * 128)) >> 4),
                                ng == 2 ? id256 : id128, k > 0);
                        else
                            tc::mma_ts_warp(tmem + 128 * buf, tmem + Sh::COL_Q + 64 * g + 8 * k,
                                            kd + ko, id128, k > 0);
                    }
                    tc::commit_warp(s_bar(SUMS ? buf : 2 * g + (turn[g]++ & 1)));
                    if (SUMS || g == ng - 1)
                        tc::commit_warp(empty_bar(sl));
                    if (i == w.te - w.tb - 1)
                        tc::commit_warp(free_bar(g));
                }
            }
        }
        if (!ok && lane == 0)
            give_up();
        // no MMA may still run when TMEM is freed
        tc::commit_warp(drain_bar);
        if (!wait_all(drain_bar, 0) && lane == 0)
            give_up();
    } else {
        // Sets of four warps: of query tile grp, pass 1 takes keys 64 half .. + 63 of every key
        // tile, pass 2 every other key tile.
        const int set = (warp - 2) >> 2, grp = set >> 1, half = set & 1;
        const int q4 = warp & 3;                          // TMEM lane quarter of this warp
        const int rr = q4 * 32 + lane;                    // this thread's TMEM lane
        const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
        const float sl2 = p.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        bool ok = true;
        int it = 0;                                       // key tiles so far
        int turn = 0;                                     // of this set's
        int units = 0;                                    // this query tile's (pass 2: all) so far
        int met = 0;
        // the query tile's threads meet; bounded, since a warp that gave up does not come
        auto meet = [&]() {
            mbar_arrive(group_bar(grp));
            return __all_sync(FULL, mbar_wait_bounded(group_bar(grp), met++ & 1));
        };
        for (; ok && w.valid; w.next(p, TPB)) {
            const int ng = groups();
            if (!SUMS && grp >= ng)
                continue;
            const int t0 = w.b * TPB + grp * TPG;         // the tile's first chunk token
            // ---- query rows ----
            // Row r = (token t0 + r / G, head r % G); rows past the chunk and those that do not
            // fill a token are zero.  The products of the piece before have ended.
            const T *qg = static_cast<const T *>(p.q);
            const int tok = t0 + rr / G;
            const bool row_valid = rr < TPG * G && tok < w.x.c;
            const int unit = (w.s * Hkv + w.h) * p.row_blocks + w.b - p.block0;
            // a piece's statistics: [half of the key tiles][query tile][row]
            float2 *stats = p.stats + (size_t)unit * (2 * ROWS) + grp * Sh::BM + rr;
            float m = -INFINITY, l = 0.f;
            auto free_rows = [&]() {
                const int n = units++;
                return n == 0 || __all_sync(FULL, mbar_wait_bounded(free_bar(SUMS ? 0 : grp),
                                                                    (n - 1) & 1));
            };
            if (!SUMS) {
                // to tensor memory, a thread 64 channels of its lane's row
                ok = free_rows();
                if (!ok)
                    break;
                if (half < D / 64) {
                    uint32_t x[32];
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        qg + ((size_t)(w.x.qs + (row_valid ? tok : 0)) * Hq + w.h * G + rr % G) * D +
                        64 * half);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 y = row_valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                        x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
                    }
                    __syncwarp();
                    tc::tmem_st32(tl + Sh::COL_Q + 64 * grp + 32 * half, x);
                }
                tc::fence_before_sync();
                mbar_arrive(q_bar(grp));
            } else {
                // to shared memory: K-major, 128-byte swizzle
                constexpr int CPR = D / 8, RSTEP = 256 / CPR, NPT = Sh::BM / RSTEP;
                const int lt = (tid - 64) & 255, ch = lt % CPR, hf = ch >> 3, c8 = ch & 7;
                uint4 qv[NPT];
#pragma unroll
                for (int i = 0; i < NPT; ++i) {
                    const int r = lt / CPR + i * RSTEP, rt = t0 + r / G;
                    qv[i] = make_uint4(0, 0, 0, 0);
                    if (r < TPG * G && rt < w.x.c)
                        qv[i] = __ldg(reinterpret_cast<const uint4 *>(
                            qg + ((size_t)(w.x.qs + rt) * Hq + w.h * G + r % G) * D + ch * 8));
                }
                // Minus log2 of the row's sum over the unit's pieces (rows that are none: -inf): by
                // the first set, or, with many pieces, by both; eight loads in flight, the first
                // of them with the queries'.
                if (units == 0)
                    grid_dependency_wait();
                constexpr int NF = 8;
                const int k0 = w.first / R, pieces = (w.first + w.nt - 1) / R - k0 + 1;
                const bool both = 2 * pieces > NF;
                const int n = !row_valid ? 0 : both ? pieces : half ? 0 : 2 * pieces;
                const int step = both ? 2 * ROWS : ROWS;
                const float2 *from = stats + (size_t)(2 * k0 + half) * ROWS;
                float2 a[NF];
                auto fetch = [&](int j) {
#pragma unroll
                    for (int i = 0; i < NF; ++i)
                        a[i] = j + i < n ? __ldcg(from + (size_t)(j + i) * step)
                                         : make_float2(-INFINITY, 0.f);
                };
                fetch(0);
                ok = free_rows();
                if (!ok)
                    break;
#pragma unroll
                for (int i = 0; i < NPT; ++i) {
                    const int r = grp * Sh::BM + lt / CPR + i * RSTEP;
                    *reinterpret_cast<uint4 *>(smem + hf * (256 * 128) + r * 128 +
                                               ((c8 ^ (r & 7)) << 4)) = qv[i];
                }
                fence_proxy_async_shared();
                mbar_arrive(q_bar(0));
                for (int j = 0; j < n; j += NF) {
                    if (j)
                        fetch(j);
#pragma unroll
                    for (int i = 0; i < NF; ++i) {
                        const float nM = fmaxf(m, a[i].x);
                        if (nM > -INFINITY)
                            l = l * exp2f(m - nM) + a[i].y * exp2f(a[i].x - nM);
                        m = nM;
                    }
                }
                // (two buffers: a thread still at the piece before reads the other)
                float *at = lse + (units & 1) * ROWS + grp * Sh::BM + rr;
                float mine = l > 0.f ? m + log2f(l) : -INFINITY;
                if (both) {
                    if (half)
                        *at = mine;
                    ok = meet();
                    const float other = *at, top = fmaxf(mine, other);
                    if (row_valid)
                        mine = top + log2f(exp2f(mine - top) + exp2f(other - top));
                }
                if (!half)
                    *at = row_valid ? -mine : -INFINITY;
                ok = ok && meet();
                if (!ok)
                    break;
            }
            // pass 2: one row block of the chunk makes the whole mass, the second query tile's
            // threads adding the first one's sums; of several each leaves its sums
            const bool alone = p.all_blocks == 1;
            float *sums = (alone ? p.mass + (size_t)(w.s * Hkv + w.h) * p.max_blocks * kBlockSize
                                 : p.sums + (size_t)(2 * unit + grp) * p.max_blocks * kBlockSize) + rr;
            // a key of the second query tile's threads that waits for the first one's sum: it is
            // there two tiles later, without delay
            float due_sum = 0.f;
            auto settle = [&](int i) {
                const int place = 2 * half + (turn & 1);
                if (!__all_sync(FULL, mbar_wait_bounded(sum_bar(place), turn >> 1 & 1)))
                    return false;
                ++turn;
                const int k0 = tile(i) * Sh::BN;
                if (k0 + rr < w.x.L)
                    sums[k0] = due_sum + part[place * Sh::BN + rr];
                return true;
            };
            const bool settles = SUMS && alone && ng == 2 && grp == 1;
            const int first_pos = w.x.L - w.x.c + t0;     // of the tile's first token
            for (int i = 0; i < w.te - w.tb; ++i, ++it) {
                const int k0 = tile(i) * Sh::BN;
                int buf, bar, phase;
                if (SUMS) {
                    buf = bar = it & 1;
                    phase = it >> 1;
                    if (buf != half)                      // the other set's
                        continue;
                    if (settles && i >= 2 && !settle(i - 2)) {
                        ok = false;
                        break;
                    }
                } else {
                    buf = ng == 2 ? (2 * i + grp) % 3 : i & 1;
                    bar = 2 * grp + (turn & 1);
                    phase = turn++ >> 1;
                }
                if (__any_sync(FULL, *abort_flag != 0) ||
                    !__all_sync(FULL, mbar_wait_bounded(s_bar(bar), phase & 1))) {
                    ok = false;
                    break;
                }
                if (grp >= ng) {                          // pass 2, one query tile
                    mbar_arrive(read_bar(buf));
                    continue;
                }
                tc::fence_after_sync();
                // columns at a time: keys for pass 1, rows for pass 2 (32: with 64 it spills)
                constexpr int CW = SUMS ? 32 : 64;
                const int c0 = SUMS ? 0 : 64 * half;
                const uint32_t tg = tl + (SUMS ? 256 * buf + 128 * grp : 128 * buf);
                // rows: keys [0, vis] of the tile are visible; keys: columns [first, 128) see it
                const int vis = row_valid ? first_pos + rr / G - k0 : -1;
                const int first = min(max(k0 + rr - first_pos, 0), 128) * G;
                const bool full = __all_sync(FULL, SUMS ? first <= 0 : vis >= c0 + 63);
                float sum = 0.f, old = 0.f;
                if (SUMS && alone && grp == ng - 1 && k0 + rr < w.x.L - w.x.c && p.decay != 0.f)
                    old = __ldcg(sums + k0);
#pragma unroll 1
                for (int c = c0; c < (SUMS ? 128 : c0 + 64); c += CW) {
                    uint32_t v[CW];
                    __syncwarp();
                    if constexpr (SUMS)
                        tc::tmem_ld32(tg + c, v);
                    else
                        tc::tmem_ld64(tg + c, v);
                    if (!SUMS || c == 128 - CW) {
                        tc::fence_before_sync();
                        mbar_arrive(read_bar(buf));
                    }
                    if (!full) {
#pragma unroll
                        for (int e = 0; e < CW; ++e)
                            if (SUMS ? e < first - c : e > vis - c)
                                v[e] = __float_as_uint(-INFINITY);
                    }
                    float mref = 0.f;
                    if constexpr (!SUMS) {
                        float mx[4];
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            auto x = [&](int q) { return __uint_as_float(v[q]); };
                            float t = fmax3(x(a), x(a + 4), x(a + 8));
#pragma unroll
                            for (int q = a + 12; q < 60; q += 8)
                                t = fmax3(t, x(q), x(q + 4));
                            mx[a] = fmaxf(t, x(a + 60));
                        }
                        const float mt =
                            fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sl2;    // scale > 0
                        if (mt > m) {
                            l *= ex2_approx(m - mt);
                            m = mt;
                        }
                        mref = m == -INFINITY ? 0.f : m;  // nothing seen yet: weights of zero
                    }
                    uint64_t sum2[4] = {0, 0, 0, 0};
                    const uint64_t nm2 = f2_pack(-mref, -mref);
                    const float4 *ls = reinterpret_cast<const float4 *>(
                        lse + (units & 1) * ROWS + grp * Sh::BM + c);
#pragma unroll
                    for (int e = 0; e < CW; e += 4) {
                        uint64_t na = nm2, nb = nm2;
                        if (SUMS) {
                            const float4 x = ls[e / 4];
                            na = f2_pack(x.x, x.y);
                            nb = f2_pack(x.z, x.w);
                        }
                        float y0, y1, y2, y3;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                         sl2x2, na),
                                  y0, y1);
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e + 2]),
                                                 __uint_as_float(v[e + 3])),
                                         sl2x2, nb),
                                  y2, y3);
                        const int o = (e >> 2) & 1;
                        sum2[o] = f2_add(sum2[o], f2_pack(ex2_approx(y0), ex2_approx(y1)));
                        sum2[2 + o] = f2_add(sum2[2 + o], f2_pack(ex2_approx(y2), ex2_approx(y3)));
                    }
                    float a, b;
                    f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), a, b);
                    sum += a + b;
                }
                if (!SUMS) {
                    l += sum;
                } else if (!alone) {
                    if (k0 + rr < w.x.L)
                        sums[k0] = sum;
                } else {
                    // Two places in turn: a set that is two of its tiles on has the other set of
                    // this buffer past the tile between, and so this one settled.
                    sum = fmaf(old, p.decay, sum);
                    if (ng == 2 && grp == 0) {
                        const int place = 2 * half + (turn++ & 1);
                        part[place * Sh::BN + rr] = sum;
                        mbar_arrive(sum_bar(place));
                    } else if (ng == 2) {
                        due_sum = sum;
                    } else if (k0 + rr < w.x.L) {
                        sums[k0] = sum;
                    }
                }
            }
            // the set's last tile of the piece, if it has one
            const int last = w.te - w.tb - 1 - ((it - 1 - half) & 1);
            if (ok && settles && last >= 0 && !settle(last)) {
                ok = false;
                break;
            }
            if (ok && !SUMS)
                stats[(size_t)blockIdx.x * (2 * ROWS) + half * ROWS] = make_float2(m, l);
        }
        if (!ok)
            give_up();
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
    // Pass 2 does not end before pass 1, also where no block of it had anything to wait for:
    // what comes next waits for pass 2 alone.
    if (SUMS)
        grid_dependency_wait();
}

// ---------------------------------------------------------------------------
// A chunk of at most 16 (token, head) rows a kv head: a query tile of 128 would be mostly empty,
// and the scores are fewer bytes than the keys, so they are kept and the keys read once.
// The warps take equal shares of the list of (sequence, kv head, 32 keys): keys are the rows
// of mma.sync's A operand, loaded 16 bytes a lane straight into fragments, the chunk's rows are
// its columns.  A lane keeps the maximum and sum of its own keys for each of its columns; a
// warp's piece of a (sequence, kv head) leaves them in slot (run + warp), which no two pieces
// share.  HBM bounds it: 4 rows over 8 sequences of 16K tokens, 8 kv heads x 128, 268 MB of keys
// and 17 MB of scores in 46 us, 6.2 TB/s; the sum of the weights takes 11 more.
// ---------------------------------------------------------------------------
constexpr int kFewThreads = kMassFewThreads, kFewKeys = 32;

// The (sequence, kv head)'s units of 32 keys, none where there is nothing to do.
__device__ __forceinline__ int few_units(const MassSeq &x)
{
    return x.blocks ? (x.L + kFewKeys - 1) / kFewKeys : 0;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kFewThreads, NT == 1 ? 4 : 3)
prefill_mass_few_kernel(const PrefillMassParams p)
{
    using M = Mma<T>;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int NI = D / 32;
    __shared__ RaggedSmem sm;
    const int lane = threadIdx.x & 31, r = lane >> 2, qd = lane & 3;
    const int warps = gridDim.x * (kFewThreads / 32);
    const int me = blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5);
    const int Hkv = p.num_kv_heads, Hq = p.num_heads, G = Hq / Hkv, n = p.num_seqs;
    const int T16 = p.max_blocks * kBlockSize, cols = p.few_cols;
    // (the sum is not started early: its blocks beside these cost 6 to 8 us where there are 9 to
    // 16 columns, 4 x 2048 keys 20.4 against 12.6, and save nothing with fewer)
    grid_dependency_wait();
    ragged_prefix<kFewThreads>(sm, 0, n, [&](int s) {
        return few_units(mass_seq(p, s, p.few_tokens, blockIdx.x == 0));
    });
    const long long total = (long long)sm.pre[n] * Hkv;
    const long long share = (total + warps - 1) / warps;
    long long u = me * share;
    const long long end = min(total, u + share);
    if (u >= end)
        return;
    int i = ragged_find(sm, n, (int)(u / Hkv));
    int nu = sm.pre[i + 1] - sm.pre[i];
    int h = (int)((u - (long long)sm.pre[i] * Hkv) / nu);
    int t = (int)((u - (long long)sm.pre[i] * Hkv) % nu);
    MassSeq x = mass_seq(p, i, p.few_tokens, false);
    // the pool tiles of blocks 2 t and 2 t + 1; past the end the last block again
    auto tiles_of = [&](int (&tile)[2]) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            int phys = __ldg(p.block_tables + (size_t)i * p.max_blocks +
                             min(2 * t + a, (x.L - 1) / kBlockSize));
            if ((unsigned)phys >= (unsigned)p.num_blocks) {
                record_error(p.err, PA_DEVERR_TABLE_RANGE);
                phys = 0;
            }
            tile[a] = phys * Hkv + h;
        }
    };
    const T *kp = static_cast<const T *>(p.k_cache);
    uint4 q[NT][NI];
    int lim[NT][2];                               // the last key that this lane's columns see
    float m[NT][2], l[NT][2];
    bool fresh = true;
    int tile[2], next[2] = {0, 0};
    tiles_of(tile);
    for (; u < end; ++u) {
        const int run = i * Hkv + h, L = x.L, key0 = kFewKeys * t;
        if (fresh) {
            const int rows = x.c * G;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int row = 8 * j + r;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const T *>(p.q) +
                    ((size_t)(x.qs + (row < rows ? row / G : 0)) * Hq + h * G + row % G) * D) + qd;
#pragma unroll
                for (int k = 0; k < NI; ++k)
                    q[j][k] = row < rows ? __ldg(src + 4 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = 8 * j + 2 * qd + e;
                    lim[j][e] = col < rows ? L - x.c + col / G : -1;
                    m[j][e] = -INFINITY;
                    l[j][e] = 0.f;
                }
            }
            fresh = false;
        }
        uint4 k4[2][2][NI];                       // [block][rows r, r + 8]
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int k = 0; k < NI; ++k)
                    k4[b][a][k] = __ldg(reinterpret_cast<const uint4 *>(
                                            kp + ((size_t)tile[b] * kBlockSize + r + 8 * a) * D) +
                                        4 * k + qd);
        bool leave = false;                       // the piece ends
        if (++t == nu) {
            t = 0;
            leave = true;
            if (++h == Hkv) {
                h = 0;
                do
                    ++i;
                while (i < n && sm.pre[i + 1] == sm.pre[i]);
                if (i < n) {
                    nu = sm.pre[i + 1] - sm.pre[i];
                    x = mass_seq(p, i, p.few_tokens, false);
                }
            }
        }
        if (u + 1 < end) {
            tiles_of(next);
            // the next 32 keys on their way to L2: two lines a lane
            constexpr int LINES = kBlockSize * D * 2 / 128;
#pragma unroll
            for (int a = 0; a < 2; ++a)
                for (int o = lane; o < LINES; o += 32)
                    prefetch_l2(kp + (size_t)next[a] * kBlockSize * D + 64 * o);
        }
        float s4[2][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s4[b][j][e] = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const uint4 &y = k4[b][0][k], &z = k4[b][1][k];
                const uint32_t a0[4] = {y.x, z.x, y.y, z.y}, a1[4] = {y.z, z.z, y.w, z.w};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    M::run(s4[b][j], a0, q[j][k].x, q[j][k].y);
                    M::run(s4[b][j], a1, q[j][k].z, q[j][k].w);
                }
            }
        float *dst = p.sums + ((size_t)run * T16 + key0 + r) * cols + 2 * qd;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // (row r, columns 2 qd and + 1), (row r + 8, the same)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s4[b][j][e] = key0 + 16 * b + r + 8 * (e >> 1) <= lim[j][e & 1]
                                      ? s4[b][j][e] * p.scale_log2
                                      : -INFINITY;
                if (8 * j + 2 * qd < cols && key0 + 16 * b < L) {
                    float *at = dst + (size_t)(16 * b) * cols + 8 * j;
                    *reinterpret_cast<float2 *>(at) = make_float2(s4[b][j][0], s4[b][j][1]);
                    *reinterpret_cast<float2 *>(at + 8 * cols) =
                        make_float2(s4[b][j][2], s4[b][j][3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float y0 = s4[0][j][e], y1 = s4[0][j][2 + e], y2 = s4[1][j][e],
                            y3 = s4[1][j][2 + e];
                const float mx = fmaxf(fmaxf(y0, y1), fmaxf(y2, y3));
                if (mx > m[j][e]) {
                    l[j][e] *= ex2_approx(m[j][e] - mx);
                    m[j][e] = mx;
                }
                const float mr = m[j][e] == -INFINITY ? 0.f : m[j][e];
                l[j][e] += (ex2_approx(y0 - mr) + ex2_approx(y1 - mr)) +
                           (ex2_approx(y2 - mr) + ex2_approx(y3 - mr));
            }
        }
        if (leave || u + 1 == end) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = m[j][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
                    float sum = top > -INFINITY ? l[j][e] * ex2_approx(m[j][e] - top) : 0.f;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        sum += __shfl_xor_sync(FULL, sum, o);
                    if (r == 0)
                        p.stats[(size_t)(run + me) * kMassFewRows + 8 * j + 2 * qd + e] =
                            make_float2(top, sum);
                }
            fresh = true;
        }
        tile[0] = next[0];
        tile[1] = next[1];
    }
}

// The weights from the kept scores: a block 1024 tokens of a (sequence, kv head), whose
// pieces' statistics its threads fold first; a warp 128 of them, four a lane.
__global__ void __launch_bounds__(kMassFinishThreads)
prefill_mass_few_finish_kernel(const PrefillMassParams p)
{
    constexpr int NTH = kMassFinishThreads, TOK = NTH / 32 * 128, ROWS = kMassFewRows;
    constexpr int PARTS = NTH / ROWS;
    __shared__ RaggedSmem units, blocks;
    __shared__ float2 part[PARTS][ROWS], fin[ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv, n = p.num_seqs, cols = p.few_cols;
    const int T16 = p.max_blocks * kBlockSize;
    grid_dependents_launch();
    grid_dependency_wait();
    ragged_prefix<NTH>(units, 0, n, [&](int s) {
        return few_units(mass_seq(p, s, p.few_tokens, false));
    });
    ragged_prefix<NTH>(blocks, 0, n, [&](int s) {
        const MassSeq x = mass_seq(p, s, p.few_tokens, false);
        return x.blocks ? (x.L + TOK - 1) / TOK : 0;
    });
    const long long all = (long long)units.pre[n] * Hkv;
    const long long share = (all + p.few_warps - 1) / p.few_warps;
    const long long total = (long long)blocks.pre[n] * Hkv;
    for (long long u = blockIdx.x; u < total; u += gridDim.x) {
        const int i = ragged_find(blocks, n, (int)(u / Hkv));
        const int nt = blocks.pre[i + 1] - blocks.pre[i];
        const int at = (int)(u - (long long)blocks.pre[i] * Hkv);
        const int h = at / nt, t0 = at % nt * TOK + 128 * warp + lane;
        const MassSeq x = mass_seq(p, i, p.few_tokens, false);
        const int run = i * Hkv + h, rows = x.c * G;
        // the old masses and the first scores while the statistics meet
        float *mass = p.mass + (size_t)run * T16 + t0;
        const float2 *y = reinterpret_cast<const float2 *>(p.sums + ((size_t)run * T16 + t0) * cols);
        float old[4], sum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            old[k] = t0 + 32 * k < x.L - x.c && p.decay != 0.f ? __ldcg(mass + 32 * k) : 0.f;
            sum[k] = 0.f;
        }
        // ---- the pieces' statistics ----
        const int nu = units.pre[i + 1] - units.pre[i];
        const long long first = (long long)units.pre[i] * Hkv + (long long)h * nu;
        const int p0 = (int)(first / share), p1 = (int)((first + nu - 1) / share);
        const int col = tid % ROWS;
        float m = -INFINITY, l = 0.f;
        if (col < rows)
            for (int j = p0 + tid / ROWS; j <= p1; j += PARTS) {
                const float2 z = __ldcg(p.stats + (size_t)(run + j) * ROWS + col);
                const float nm = fmaxf(m, z.x);
                if (nm > -INFINITY)
                    l = l * exp2f(m - nm) + z.y * exp2f(z.x - nm);
                m = nm;
            }
        part[tid / ROWS][col] = make_float2(m, l);
        __syncthreads();
        if (tid < ROWS) {
            float top = -INFINITY, s = 0.f;
#pragma unroll
            for (int j = 0; j < PARTS; ++j)
                top = fmaxf(top, part[j][tid].x);
#pragma unroll
            for (int j = 0; j < PARTS; ++j)
                s += part[j][tid].x > -INFINITY ? part[j][tid].y * exp2f(part[j][tid].x - top) : 0.f;
            fin[tid] = tid < rows ? make_float2(top, 1.f / s) : make_float2(0.f, 0.f);
        }
        __syncthreads();
        // ---- the sums ----
        for (int g = 0; g < cols; g += 4) {
            float2 v[4][2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k][e] = t0 + 32 * k < x.L && g + 2 * e < cols
                                  ? __ldcg(y + (16 * k * cols + g / 2 + e))
                                  : make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 a = fin[min(g + 2 * e, ROWS - 2)], b = fin[min(g + 2 * e, ROWS - 2) + 1];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sum[k] = fmaf(ex2_approx(v[k][e].x - a.x), a.y,
                                  fmaf(ex2_approx(v[k][e].y - b.x), b.y, sum[k]));
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (t0 + 32 * k < x.L)
                mass[32 * k] = fmaf(old[k], p.decay, sum[k]);
        __syncthreads();                          // part and fin are written again
    }
}

// ---------------------------------------------------------------------------
// The same for short sequences in one launch: a thread block takes a (sequence,
// kv head) whole, its warps 16 (token, head) rows at a time with mma.sync.  The
// channels of a product may be taken in any order, so rows of q and k are
// loaded 16 bytes a lane straight into fragments.  Where the rows are few, the keys are
// split between the warps, which exchange their rows' statistics; the warps' sums for a
// key meet in shared memory.  What bounds it is one block's chain: lengths, table, rows,
// then 1.0 us (64 channels) or 1.3 us (128) for every 32 keys of a warp and pass.  Two chunks
// of 5 and 70 tokens, 8/2 heads x 64, the long one over 70 keys 10.3 us in a graph (by the passes
// and their sum 13.4), over 150 keys 17.9 (13.3).
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kMassShortThreads) prefill_mass_short_kernel(const PrefillMassParams p)
{
    using M = Mma<T>;
    constexpr uint32_t FULL = 0xffffffffu;
    constexpr int NW = kMassShortThreads / 32, NI = D / 32;
    constexpr int N8 = 4;                         // 8-key steps in flight
    __shared__ float acc[NW][kMassShortKeys];
    __shared__ float2 part[NW][16];
    __shared__ int tile_of[kMassShortKeys / kBlockSize];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, qd = lane & 3;
    const int Hkv = p.num_kv_heads, Hq = p.num_heads, G = Hq / Hkv;
    const int s = blockIdx.x / Hkv, h = blockIdx.x % Hkv;
    grid_dependents_launch();
    grid_dependency_wait();
    const MassSeq x = mass_seq(p, s, kMassTiles * (kMassRows / G), h == 0 && tid == 0);
    if (x.blocks == 0)
        return;
    const int nblk = (x.L + kBlockSize - 1) / kBlockSize;
    const int rows = x.c * G, steps = (x.L + 7) / 8;
    // everything that will be read is on its way to L2 before the first use waits for it
    constexpr int LPR = D * 2 / 128;              // lines of a row
    for (int i = tid; i < rows * LPR; i += kMassShortThreads)
        prefetch_l2(static_cast<const T *>(p.q) +
                    ((size_t)(x.qs + i / LPR / G) * Hq + h * G + i / LPR % G) * D + i % LPR * 64);
    float *mass = p.mass + (size_t)blockIdx.x * p.max_blocks * kBlockSize;
    if (tid * 32 < x.L)
        prefetch_l2(mass + tid * 32);
    if (tid < nblk) {
        int phys = __ldg(p.block_tables + (size_t)s * p.max_blocks + tid);
        if ((unsigned)phys >= (unsigned)p.num_blocks) {
            record_error(p.err, PA_DEVERR_TABLE_RANGE);
            phys = 0;
        }
        tile_of[tid] = phys * Hkv + h;
    }
    const int used = min((rows + 15) / 16, NW);   // rows of acc
    if (warp < used)
        for (int t = lane; t < nblk * kBlockSize; t += 32)
            acc[warp][t] = 0.f;
    __syncthreads();
    for (int i = tid; i < x.L * LPR; i += kMassShortThreads)
        prefetch_l2(static_cast<const T *>(p.k_cache) +
                    ((size_t)tile_of[i / LPR / kBlockSize] * kBlockSize + i / LPR % kBlockSize) * D +
                    i % LPR * 64);
    const uint4 *kp = static_cast<const uint4 *>(p.k_cache) + qd;
    // 16 rows a warp; a round that leaves warps over splits the keys of 16 rows into parts
    for (int base = 0; base < rows; base += 16 * NW) {
        const int groups = min((rows - base + 15) / 16, NW), parts = NW / groups;
        const int mine = warp / groups, row0 = base + 16 * (warp % groups);   // no part: parts on
        float *sums = acc[warp % groups];
        // rows row0 + r and + 8; past the last one that one again, without weight
        uint32_t a[2 * NI][4];
        int pos[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = min(row0 + r + 8 * e, rows - 1), tok = row / G;
            pos[e] = row0 + r + 8 * e < rows ? x.L - x.c + tok : -1;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                                   static_cast<const T *>(p.q) +
                                   ((size_t)(x.qs + tok) * Hq + h * G + row % G) * D) + qd;
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const uint4 y = __ldg(src + 4 * k);
                a[2 * k][e] = y.x, a[2 * k][2 + e] = y.y;
                a[2 * k + 1][e] = y.z, a[2 * k + 1][2 + e] = y.w;
            }
        }
        // f(key step, scores in base 2: two keys of two rows) for every 8 keys that a row sees
        const int seen = min(steps, (x.L - x.c + (min(row0 + 15, rows - 1)) / G) / 8 + 1);
        const int share = (seen + parts - 1) / parts;
        const int from = mine * share, last = mine < parts ? min(seen, from + share) : 0;
        auto each = [&](auto &&f) {
            for (int j0 = from; j0 < last; j0 += N8) {
                uint4 b[N8][NI];
#pragma unroll
                for (int i = 0; i < N8; ++i) {
                    const int t = min(8 * (j0 + i) + r, x.L - 1);
                    const uint4 *src = kp + ((size_t)tile_of[t / kBlockSize] * kBlockSize +
                                             t % kBlockSize) * (D / 8);
#pragma unroll
                    for (int k = 0; k < NI; ++k)
                        b[i][k] = __ldg(src + 4 * k);
                }
#pragma unroll
                for (int i = 0; i < N8; ++i) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < NI; ++k) {
                        M::run(d, a[2 * k], b[i][k].x, b[i][k].y);
                        M::run(d, a[2 * k + 1], b[i][k].z, b[i][k].w);
                    }
                    // d: (row r, keys 2 qd and + 1), (row r + 8, the same)
                    const int t = 8 * (j0 + i) + 2 * qd;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        d[e] = t + (e & 1) <= pos[e >> 1] ? d[e] * p.scale_log2 : -INFINITY;
                    if (j0 + i < last)
                        f(j0 + i, d);
                }
            }
        };
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        each([&](int, const float (&d)[4]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mx = fmaxf(d[2 * e], d[2 * e + 1]);
                if (mx > m[e]) {
                    l[e] *= exp2f(m[e] - mx);
                    m[e] = mx;
                }
                if (m[e] > -INFINITY)
                    l[e] += exp2f(d[2 * e] - m[e]) + exp2f(d[2 * e + 1] - m[e]);
            }
        });
        // the row's four lanes
        float top[2], inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[e] = m[e];
#pragma unroll
            for (int off = 1; off < 4; off <<= 1)
                top[e] = fmaxf(top[e], __shfl_xor_sync(FULL, top[e], off));
            inv[e] = m[e] > -INFINITY ? l[e] * exp2f(m[e] - top[e]) : 0.f;
#pragma unroll
            for (int off = 1; off < 4; off <<= 1)
                inv[e] += __shfl_xor_sync(FULL, inv[e], off);
        }
        if (parts > 1) {                          // (the last round alone)
            if (mine < parts && qd == 0) {
                part[warp][r] = make_float2(top[0], inv[0]);
                part[warp][r + 8] = make_float2(top[1], inv[1]);
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float M = -INFINITY, sum = 0.f;
                for (int i = 0; i < parts; ++i)
                    M = fmaxf(M, part[warp % groups + i * groups][r + 8 * e].x);
                for (int i = 0; i < parts; ++i) {
                    const float2 y = part[warp % groups + i * groups][r + 8 * e];
                    sum += y.x > -INFINITY ? y.y * exp2f(y.x - M) : 0.f;
                }
                top[e] = M;
                inv[e] = sum;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            inv[e] = pos[e] >= 0 ? 1.f / inv[e] : 0.f;
            top[e] = pos[e] >= 0 ? top[e] : 0.f;
        }
        each([&](int j, const float (&d)[4]) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[e] = exp2f(d[e] - top[0]) * inv[0] + exp2f(d[2 + e] - top[1]) * inv[1];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    w[e] += __shfl_xor_sync(FULL, w[e], off);
            }
            if (r == 0) {
                sums[8 * j + 2 * qd] += w[0];
                sums[8 * j + 2 * qd + 1] += w[1];
            }
        });
    }
    __syncthreads();
    for (int t = tid; t < x.L; t += kMassShortThreads) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            sum += w < used ? acc[w][t] : 0.f;
        mass[t] = add_mass(mass + t, p.decay, t >= x.L - x.c, sum);
    }
}

// Several row blocks: the sum over a sequence's query tiles of the launch, added to the mass (to
// what the launches before made of it, from the second on).  Eight warps
// (with two row blocks, four) share out the query tiles of 128 tokens of a (sequence, kv
// head), four tokens a lane.  What bounds it is a warp's chain of loads: 14 runs to
// 1130 tokens, 34 row blocks, 9 us (a warp for all of the tiles 25); 64 runs to 5534 tokens, 2 row
// blocks, 51 us in all with four warps, 54 with eight.
__global__ void __launch_bounds__(kMassFinishThreads)
prefill_mass_finish_kernel(const PrefillMassParams p)
{
    constexpr int NTH = kMassFinishThreads, NW = NTH / 32, TOK = 128;
    __shared__ RaggedSmem sm;
    __shared__ float4 part[NW][TOK / 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int split = p.row_blocks == 2 ? 4 : NW;
    const int Hkv = p.num_kv_heads, G = p.num_heads / Hkv, TPG = kMassRows / G;
    const int T = p.max_blocks * kBlockSize;
    grid_dependents_launch();
    grid_dependency_wait();
    for (int begin = 0; begin < p.num_seqs; begin += kRaggedSeqs) {
        const int n = min(kRaggedSeqs, p.num_seqs - begin);
        ragged_prefix<NTH>(sm, begin, n, [&](int s) {
            // what the passes skipped stays as it was
            const MassSeq x = mass_seq(p, s, kMassTiles * TPG, false);
            return x.blocks > p.block0 ? (x.L + TOK - 1) / TOK : 0;
        });
        const long long total = (long long)sm.pre[n] * Hkv;
        for (long long u0 = (long long)blockIdx.x * (NW / split); u0 < total;
             u0 += (long long)gridDim.x * (NW / split)) {
            // (past the end the last unit again, which is not written)
            const long long u = min(u0 + warp / split, total - 1);
            const int i = ragged_find(sm, n, (int)(u / Hkv));
            const int nt = sm.pre[i + 1] - sm.pre[i];
            const int at = (int)(u - (long long)sm.pre[i] * Hkv);
            const int s = begin + i, h = at / nt, t0 = at % nt * TOK, t = t0 + 4 * lane;
            const int L = __ldg(p.seq_lens + s);
            const int c = __ldg(p.query_start + s + 1) - __ldg(p.query_start + s);
            const size_t run = (size_t)s * Hkv + h;
            const float *from = p.sums + run * (kMassTiles * p.row_blocks) * T + t;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            // query tiles whose keys reach t (a unit's end where its last row's do)
            const int TPB = kMassTiles * TPG, k0 = kMassTiles * p.block0;
            const int tiles = t < L ? min((c + TPG - 1) / TPG, k0 + kMassTiles * p.row_blocks) : 0;
#pragma unroll 4
            for (int k = max(p.block0, (t - (L - c)) / TPB) * kMassTiles + warp % split; k < tiles;
                 k += split) {
                const float4 x =
                    __ldcg(reinterpret_cast<const float4 *>(from + (size_t)(k - k0) * T));
                const int end = L - c + min((k / kMassTiles + 1) * TPB, c);
                sum.x += x.x;                     // (t itself is reached by the first unit)
                sum.y += t + 1 < end ? x.y : 0.f;
                sum.z += t + 2 < end ? x.z : 0.f;
                sum.w += t + 3 < end ? x.w : 0.f;
            }
            part[warp][lane] = sum;
            __syncthreads();
            // a warp's share of the 128 tokens
            const int j = warp % split * (TOK / split) + lane;
            if (lane < TOK / split && t0 + j < L && u0 + warp / split < total) {
                float all = 0.f;
                for (int w = 0; w < split; ++w)
                    all += reinterpret_cast<const float *>(part[warp / split * split + w])[j];
                float *mass = p.mass + run * T + t0 + j;
                *mass = p.block0 ? *mass + all : add_mass(mass, p.decay, t0 + j >= L - c, all);
            }
            __syncthreads();
        }
    }
}

template <typename T, int D>
void fill(MassKernels *k)
{
    k->stats = reinterpret_cast<const void *>(&prefill_mass_kernel<T, D, false>);
    k->sums = reinterpret_cast<const void *>(&prefill_mass_kernel<T, D, true>);
    k->whole = reinterpret_cast<const void *>(&prefill_mass_short_kernel<T, D>);
    k->few[0] = reinterpret_cast<const void *>(&prefill_mass_few_kernel<T, D, 1>);
    k->few[1] = reinterpret_cast<const void *>(&prefill_mass_few_kernel<T, D, 2>);
    k->few_finish = reinterpret_cast<const void *>(&prefill_mass_few_finish_kernel);
    k->threads = MassShape<D, false>::THREADS;
    k->smem_stats = MassShape<D, false>::SMEM;
    k->smem_sums = MassShape<D, true>::SMEM;
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
