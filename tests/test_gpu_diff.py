"""diff_decode and diff_prefill against the formula in 64 bits (diff_util: the
tolerance and its derivation).  Pool slots that hold no live token are NaN."""
import math

import numpy as np
import pytest
import torch

from diff_util import assert_close, reference
from gpu_util import TORCH_DTYPE
from paged_kv_cache_260_gb300.block_manager import BlockManager

pytestmark = pytest.mark.gpu

EPS = 1e-5
# what rounds a softmax weight: the decode of groups of up to 8 heads keeps a rounded weight's
# rest (half a step of half a step), the prefill and the decode of wider groups do not
P_DECODE = {"f16": 2.0 ** -21, "bf16": 2.0 ** -17}
P_PREFILL = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def p_round(decode, dtype, group):
    return (P_DECODE if decode and group <= 8 else P_PREFILL)[dtype]


class Pool:
    def __init__(self, lens, hq, hkv, d, dtype, chunks=None, norm=True, seed=0, maxb=None,
                 gain=2.0, out_scale=0.4):
        g = torch.Generator().manual_seed(seed)
        dt = TORCH_DTYPE[dtype]
        self.dtype, self.lens_h, n = dtype, list(lens), len(lens)
        used = [(x + 15) // 16 for x in lens]
        nb = sum(used) + 3
        mb = maxb or max(1, max(used, default=0))
        order = torch.randperm(nb, generator=g)
        self.tables_h = torch.full((n, mb), -1, dtype=torch.int32)
        at = 0
        self.k_h, self.v_h = (torch.full((nb, hkv, 16, d), float("nan"), dtype=dt)
                              for _ in range(2))
        for s, x in enumerate(lens):
            for b in range(used[s]):
                blk = int(order[at + b])
                self.tables_h[s, b] = blk
                live = min(16, x - 16 * b)
                self.k_h[blk, :, :live] = torch.randn(hkv, live, d, generator=g).to(dt)
                self.v_h[blk, :, :live] = torch.randn(hkv, live, d, generator=g).to(dt)
            at += used[s]
        self.k, self.v, self.tables = self.k_h.cuda(), self.v_h.cuda(), self.tables_h.cuda()
        self.lens = torch.tensor(self.lens_h, dtype=torch.int32).cuda()
        self.chunks = chunks
        rows = n if chunks is None else sum(chunks)
        self.q_h = (gain * torch.randn(rows, hq, d, generator=g)).to(dt)
        self.q = self.q_h.cuda()
        self.lam = torch.rand(hq, generator=g).mul(1.2).cuda()
        self.w = (1 + 0.3 * torch.randn(d, generator=g)).to(dt).cuda() if norm else None
        self.scale, self.out_scale = (d // 2) ** -0.5, out_scale
        self.out = torch.full((rows + 2, hq, d), 7.0, dtype=dt, device="cuda")
        if chunks is not None:
            self.start_h = [0] + np.cumsum(chunks).tolist()
            self.start = torch.tensor(self.start_h, dtype=torch.int32).cuda()

    def decode(self, pa, out=None, **kw):
        out = self.out[:len(self.lens_h)] if out is None else out
        pa.diff_decode(out, self.q, self.k, self.v, self.tables, self.lens, self.lam, self.scale,
                       norm_weight=self.w, eps=EPS, out_scale=self.out_scale, **kw)
        return out

    def prefill(self, pa, out=None, longest=None, **kw):
        out = self.out[:self.start_h[-1]] if out is None else out
        pa.diff_prefill(out, self.q, self.k, self.v, self.tables, self.lens, self.start,
                        max(self.chunks) if longest is None else longest, self.lam, self.scale,
                        norm_weight=self.w, eps=EPS, out_scale=self.out_scale, **kw)
        return out

    def rows(self, s):
        """(first row, positions) of sequence s."""
        if self.chunks is None:
            return s, [self.lens_h[s] - 1]
        c = self.chunks[s]
        return self.start_h[s], list(range(self.lens_h[s] - c, self.lens_h[s]))

    def check(self, out, only=None):
        p = p_round(self.chunks is None, self.dtype, self.q_h.shape[1] // self.k_h.shape[1])
        w = None if self.w is None else self.w.cpu()
        for s in range(len(self.lens_h)) if only is None else only:
            r0, pos = self.rows(s)
            ref, tol = reference(self.q_h[r0:r0 + len(pos)], self.k_h, self.v_h, self.tables_h, s,
                                 pos, self.lam.cpu(), self.scale, w, EPS, self.out_scale, p)
            assert_close(out[r0:r0 + len(pos)], ref, tol, f"sequence {s}")
        assert bool((self.out[out.shape[0]:] == 7).all()), "rows past the last sequence"


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 257, 700, 1029]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dtype", [
    (2, 2, 64, "f16"), (8, 8, 128, "bf16"), (4, 2, 128, "f16"), (6, 2, 64, "bf16"),
    (32, 8, 128, "bf16"), (4, 1, 64, "f16"), (5, 1, 128, "f16"), (12, 2, 64, "bf16"),
    (7, 1, 64, "f16"), (16, 2, 128, "bf16"), (24, 3, 64, "f16"), (9, 1, 128, "f16"),
    (16, 1, 64, "bf16"), (26, 2, 128, "bf16"), (30, 2, 64, "f16"), (16, 1, 128, "f16")])
def test_decode_ragged(pa, hq, hkv, d, dtype, norm):
    x = Pool(LENS, hq, hkv, d, dtype, norm=norm, seed=hq + d)
    x.check(x.decode(pa))
    assert bool((x.out[0] == 0).all())                       # length 0: zeros
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 8, 64, "f16"), (8, 2, 128, "bf16"),
                                            (10, 2, 128, "f16"), (24, 2, 64, "bf16")])
@pytest.mark.parametrize("lens", [[1], [16], [100, 3, 0, 77], [128] * 4])
def test_decode_short_runs_are_not_split(pa, hq, hkv, d, dtype, lens):
    x = Pool(lens, hq, hkv, d, dtype, seed=len(lens), maxb=8)
    x.check(x.decode(pa))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype", [(4, 1, 128, "bf16"), (8, 1, 64, "f16"),
                                            (13, 1, 128, "bf16")])
def test_decode_one_long_sequence(pa, hq, hkv, d, dtype):
    x = Pool([20011], hq, hkv, d, dtype, seed=5)             # cut across every worker
    x.check(x.decode(pa))


def test_decode_large_batch(pa):
    # more sequences than the decode keeps in shared memory
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 40, 2300).tolist()
    x = Pool(lens, 4, 2, 64, "f16", seed=6)
    x.check(x.decode(pa), only=list(range(0, 2300, 97)) + [2299])
    zero = torch.tensor([i for i, n in enumerate(lens) if n == 0]).cuda()
    assert bool((x.out[zero] == 0).all())
    assert pa.get_device_error() == 0


def test_decode_empty_batch_and_all_empty(pa):
    x = Pool([0, 0, 0], 8, 2, 128, "f16")
    x.check(x.decode(pa))
    e = Pool([4], 8, 2, 128, "f16")
    pa.diff_decode(e.out[:0], e.q[:0], e.k, e.v, e.tables[:0], e.lens[:0], e.lam, 1.0)
    assert bool((e.out == 7).all())


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (12, 2, 64)])
def test_zero_lambda_is_plain_attention_of_the_first_map(pa, hq, hkv, d):
    x = Pool([40, 300, 7], hq, hkv, d, "f16", norm=False, out_scale=1.0)
    x.lam.zero_()
    got = x.decode(pa).clone()
    q = x.q.clone()
    q[..., d // 2:] = 0
    out = torch.empty_like(got)
    pa.decode(out, q, x.k, x.v, x.tables, x.lens, x.scale)
    # both are within half a step (and the weights' rounding) of the same value
    assert float((got.float() - out.float()).abs().max()) <= 4e-3
    # equal maps and a factor of one leave nothing, so the norm sees zeros
    x.k[..., d // 2:] = x.k[..., :d // 2]
    x.q[..., d // 2:] = x.q[..., :d // 2]
    x.lam.fill_(1.0)
    x.w = torch.ones(d, dtype=torch.float16, device="cuda")
    out = x.decode(pa)
    # y is at most 2 * 2^-19 of the values, |v| < 6; divided by sqrt(EPS)
    assert float(out.abs().max()) <= x.out_scale * 2 * 2.0 ** -19 * 6 / math.sqrt(EPS)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_large_scores_and_growing_maxima(pa, kind):
    # scores of about a hundred, the maximum rising along the sequence
    lens = [500, 131]
    x = Pool(lens, 8, 2, 128, "bf16", chunks=None if kind == "decode" else [70, 131], gain=8.0)
    for s, n in enumerate(lens):
        for t in range(n):
            b = int(x.tables_h[s, t // 16])
            x.k_h[b, :, t % 16] *= 0.2 + 3.0 * t / n
    x.k.copy_(x.k_h)
    x.check(x.decode(pa) if kind == "decode" else x.prefill(pa))


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dtype", [
    (2, 2, 64, "f16"), (4, 4, 128, "bf16"), (8, 2, 128, "f16"), (6, 2, 64, "bf16"),
    (10, 2, 128, "bf16"), (7, 1, 64, "f16"), (16, 1, 128, "bf16")])
@pytest.mark.parametrize("plan", [True, False])
def test_prefill_ragged(pa, hq, hkv, d, dtype, norm, plan):
    lens = [1, 16, 70, 300, 129, 128, 517, 40]
    chunks = [1, 16, 3, 140, 129, 128, 1, 0]
    x = Pool(lens, hq, hkv, d, dtype, chunks=chunks, norm=norm, seed=hq)
    x.check(x.prefill(pa, workspace="auto" if plan else None))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 128, "bf16"), (4, 4, 64, "f16")])
def test_prefill_longer(pa, hq, hkv, d, dtype):
    x = Pool([2000, 900], hq, hkv, d, dtype, chunks=[333, 900], seed=3)
    x.check(x.prefill(pa))


@pytest.mark.parametrize("plan", [True, False])
def test_prefill_more_blocks_than_sms(pa, plan):
    # enough blocks for the work order, whose K/V fits in L2
    lens = [700, 300, 128, 513, 64]
    x = Pool(lens, 16, 8, 128, "bf16", chunks=[700, 299, 128, 1, 64], seed=14)
    x.check(x.prefill(pa, workspace="auto" if plan else None))
    assert pa.get_device_error() == 0


def test_prefill_order_by_sequence(pa):
    # K/V past L2: the order goes sequence by sequence
    lens, chunks = [13000, 12001, 12500], [150, 70, 90]
    x = Pool(lens, 16, 8, 128, "bf16", chunks=chunks, seed=15)
    a = x.prefill(pa).clone()
    x.check(a, only=[1])
    assert torch.equal(x.prefill(pa, workspace=None), a)     # the order changes no result
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,chunks", [(96, [3, 1, 2]), (128, [3, 1, 2]), (128, [1, 1, 1]),
                                       (43, [7, 1, 2])])
def test_prefill_wide_groups(pa, hq, chunks):
    # one token's heads, or a few, fill a query tile
    x = Pool([200, 1, 130], hq, 1, 64, "bf16", chunks=chunks, seed=hq)
    x.check(x.prefill(pa))


@pytest.mark.parametrize("plan", [True, False])
@pytest.mark.parametrize("longest", [20, 64])
def test_prefill_longest_chunk_understated(pa, plan, longest):
    """A chunk longer than max_query_len is reported, its last rows are right, no row
    outside it is touched; the other sequences are whole."""
    x = Pool([400, 90], 8, 2, 128, "f16", chunks=[300, 15], seed=8)
    out = x.prefill(pa, longest=longest, workspace="auto" if plan else None)
    assert pa.get_device_error() == pa.DEVERR["QUERY_RANGE"]
    good = out.clone()
    x.check(x.prefill(pa))
    same = (good == out).flatten(1).all(1)
    assert bool(same[300:].all()) and bool(same[288:300].all())   # from the last whole tile on
    assert bool((good[~same] == 7).all())


def test_decode_negative_scale(pa):
    x = Pool([40, 300, 17], 8, 2, 128, "bf16", seed=12)
    x.scale = -x.scale
    x.check(x.decode(pa))


def test_prefill_rows_outside_chunks_stay(pa):
    x = Pool([50, 20], 8, 2, 64, "f16", chunks=[30, 20])
    x.prefill(pa)
    keep = x.out.clone()
    # two padding sequences without rows, and a longest chunk that none reaches
    x.lens = torch.cat([x.lens, torch.zeros(2, dtype=torch.int32, device="cuda")])
    x.start = torch.cat([x.start, x.start[-1:].repeat(2)])
    x.tables = torch.cat([x.tables, torch.full_like(x.tables, -1)])
    x.out.fill_(7.0)
    x.prefill(pa, longest=200)
    assert torch.equal(x.out, keep) and pa.get_device_error() == 0


def test_prefill_of_one_row_is_a_decode(pa):
    x = Pool([77, 300, 16], 8, 2, 128, "bf16", chunks=[1, 1, 1], seed=9)
    x.check(x.prefill(pa))
    x.chunks = None
    x.check(x.decode(pa))


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_bad_tables_and_lengths_are_reported(pa, kind):
    x = Pool([40, 60, 33], 8, 2, 128, "f16", chunks=None if kind == "decode" else [10, 60, 33])
    run = x.decode if kind == "decode" else x.prefill
    x.k.nan_to_num_(0.0)
    x.v.nan_to_num_(0.0)
    good = run(pa).clone()
    r0, pos = x.rows(1)
    keep = torch.ones(good.shape[0], dtype=torch.bool, device="cuda")
    keep[r0:r0 + len(pos)] = False
    for value in (x.k.shape[0], -3, 2 ** 31 - 1):
        x.tables[1, 2] = value
        out = run(pa).clone()
        assert pa.get_device_error() == pa.DEVERR["TABLE_RANGE"]
        assert torch.equal(out[keep], good[keep])            # the others are not touched
    x.tables.copy_(x.tables_h)
    for value in (-1, 16 * x.tables.shape[1] + 1):
        x.lens[1] = value
        out = run(pa).clone()
        assert pa.get_device_error() & pa.DEVERR["SEQLEN_RANGE"]
        assert torch.equal(out[keep], good[keep])


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_graph_replay_with_changing_inputs(pa, kind):
    mk = lambda lens, seed: Pool(lens, 8, 2, 128, "bf16",  # noqa: E731
                                 chunks=None if kind == "decode" else [9, 9, 9], seed=seed,
                                 maxb=40)
    x = mk([300, 20, 600], 1)
    run = x.decode if kind == "decode" else x.prefill
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(pa)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):                                   # back to back in one graph
            run(pa)
    g.replay()
    x.check(x.out[:x.q.shape[0]])
    y = mk([17, 620, 64], 2)
    big = torch.full((max(x.k.shape[0], y.k.shape[0]), *x.k.shape[1:]), float("nan"),
                     dtype=x.k.dtype)
    assert y.k.shape[0] <= x.k.shape[0]                      # it fits the captured pool
    for a, b in ((x.k, y.k_h), (x.v, y.v_h)):
        big[:b.shape[0]] = b
        a.copy_(big[:a.shape[0]])
    for a, b in ((x.q, y.q), (x.tables, y.tables), (x.lens, y.lens), (x.lam, y.lam), (x.w, y.w)):
        a.copy_(b)
    g.replay()
    y.check(x.out[:x.q.shape[0]])
    assert pa.get_device_error() == 0


def test_two_streams_with_workspaces_of_their_own(pa):
    xs = [Pool([900, 33, 400], 8, 2, 128, "bf16", seed=20 + i) for i in range(2)]
    want = [x.decode(pa).clone() for x in xs]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        for x, s in zip(xs, ss):
            x.decode(pa, stream=s)
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        assert torch.equal(x.out[:3], w)                     # bit-stable too


def test_scratch_comes_from_the_calls_stream(pa):
    # memory that the current stream has just freed may still be in use there
    x = Pool([900, 33], 8, 2, 128, "bf16", chunks=[100, 33], seed=23)
    y = Pool([900, 33], 8, 2, 128, "bf16", seed=23)
    s = torch.cuda.Stream()
    for make in (lambda **k: pa.diff_decode_workspace_for(y.q, y.k, y.tables, **k),
                 lambda **k: pa.diff_prefill_workspace_for(x.q, x.k, x.lens, 100, **k),
                 lambda **k: pa.workspace_for(y.q, y.k, y.tables, **k)):
        torch.cuda.synchronize()
        first = make()
        at = first.data_ptr()
        del first
        assert make().data_ptr() == at                       # the allocator does reuse it
        assert make(stream=s).data_ptr() != at


def test_offsets_past_32_bits(pa):
    # a pool of more than 2^31 elements whose live blocks lie at its end
    hkv, d = 8, 128
    nb = (2 ** 31 // (hkv * 16 * d)) + 300
    k = torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    x = Pool([100, 300], 16, hkv, d, "bf16", chunks=[20, 33], seed=30)
    small = x.k.shape[0]
    k[-small:], v[-small:] = x.k, x.v
    tables = torch.where(x.tables >= 0, x.tables + (nb - small), x.tables)
    want = x.prefill(pa).clone()
    x.k, x.v, x.tables = k, v, tables
    assert torch.equal(x.prefill(pa), want)
    y = Pool([100, 300], 16, hkv, d, "bf16", seed=30)
    want = y.decode(pa).clone()
    k[-small:], v[-small:] = y.k, y.v
    y.tables = torch.where(y.tables >= 0, y.tables + (nb - small), y.tables)
    y.k, y.v = k, v
    assert torch.equal(y.decode(pa), want)
    assert pa.get_device_error() == 0


def test_refusals(pa):
    x = Pool([40, 60], 8, 2, 128, "f16")
    ok = dict(out=x.out[:2], q=x.q, k_cache=x.k, v_cache=x.v, block_tables=x.tables,
              seq_lens=x.lens, lam=x.lam, scale=1.0)
    for kw in (dict(lam=x.lam[:4]), dict(lam=x.lam.half()), dict(lam=x.lam.cpu()),
               dict(q=x.q.bfloat16()), dict(out=x.out), dict(seq_lens=x.lens.long()),
               dict(block_tables=x.tables.long()), dict(block_tables=x.tables[:1]),
               dict(norm_weight=torch.ones(128, device="cuda")),
               dict(norm_weight=torch.ones(64, device="cuda", dtype=torch.float16)),
               dict(v_cache=x.v[:, :1]), dict(q=x.q.cpu()),
               dict(q=x.q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            pa.diff_decode(**{**ok, **kw})
    for kw in (dict(eps=-1.0, norm_weight=None), dict(scale=math.nan), dict(out_scale=math.inf)):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.diff_decode(**{**ok, **kw})
        assert e.value.status == 1
    need = pa.diff_decode_workspace_size(2, 8, 2, 128, x.tables.shape[1])
    big = Pool([400, 60], 8, 2, 128, "f16")                  # wide tables: the split needs it
    need = pa.diff_decode_workspace_size(2, 8, 2, 128, big.tables.shape[1])
    with pytest.raises(pa.PagedAttnError) as e:
        big.decode(pa, workspace=torch.empty(need - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    big.check(big.decode(pa, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")))
    g17 = Pool([40], 17, 1, 64, "f16")
    with pytest.raises(pa.PagedAttnError) as e:
        g17.decode(pa)
    assert e.value.status == 2
    torch.cuda.synchronize()
    assert bool((x.out == 7).all())                          # nothing was launched


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("f16", 6, 1, 64)])
def test_serving_flow(pa, dtype, hq, hkv, d):
    """Prompts and decode steps of a differential-attention model: rope_and_cache fills the
    pool with both keys of a head, diff_prefill attends the chunks, a sequence is forked,
    copy_blocks separates the samples, and rope_and_cache + diff_decode go on."""
    g = torch.Generator().manual_seed(40)
    dt = TORCH_DTYPE[dtype]
    nb, maxb, scale = 96, 12, (d // 2) ** -0.5
    kc, vc = (torch.randn(nb, hkv, 16, d, generator=g).to(dt).cuda() for _ in range(2))
    lam = torch.rand(hq, generator=g).cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dt).cuda()
    qn, kn = ((1.4 + 0.1 * torch.randn(d // 2, generator=g)).to(dt).cuda() for _ in range(2))
    ang = torch.arange(400).double()[:, None] * 10000.0 ** (-torch.arange(0, d // 2, 2) / (d / 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    bm = BlockManager(nb)

    def step(sids, chunks):
        """One engine step over the sequences' next tokens; checks every row."""
        slots, pairs, pos = [], [], []
        for s, c in zip(sids, chunks):
            before = bm.block_table(s, maxb)[2]
            sl, cow = bm.append(s, c)
            slots += sl.tolist()
            pos += list(range(before, before + c))
            if cow:
                pairs.append(cow)
        if pairs:
            pa.copy_blocks(kc, vc, torch.tensor(pairs).cuda())
        t = len(slots)
        qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g).to(dt).cuda()
        q, k, v = (a.view(t, -1, d) for a in qkv.split([hq * d, hkv * d, hkv * d], 1))
        qo = torch.empty(t, hq, d, dtype=dt, device="cuda")
        pa.rope_and_cache(qo, q, k, v, kc, vc, torch.tensor(slots).cuda(),
                          torch.tensor(pos).int().cuda(), cs, q_norm=qn, k_norm=kn, eps=EPS,
                          num_maps=2)
        tables = torch.from_numpy(np.stack([bm.block_table(s, maxb)[0] for s in sids]))
        lens = [bm.block_table(s, maxb)[2] for s in sids]
        out = torch.full((t, hq, d), float("nan"), dtype=dt, device="cuda")
        args = (out, qo, kc, vc, tables.cuda(), torch.tensor(lens).int().cuda())
        decode = chunks == [1] * len(sids)
        if decode:
            pa.diff_decode(*args, lam, scale, norm_weight=w, eps=EPS, out_scale=0.3)
        else:
            start = torch.tensor([0] + np.cumsum(chunks).tolist()).int().cuda()
            pa.diff_prefill(*args, start, max(chunks), lam, scale, norm_weight=w, eps=EPS,
                            out_scale=0.3)
        assert pa.get_device_error() == 0
        row = 0
        for i, (s, c) in enumerate(zip(sids, chunks)):
            p = list(range(lens[i] - c, lens[i]))
            ref, tol = reference(qo[row:row + c].cpu(), kc.cpu(), vc.cpu(), tables, i, p, lam.cpu(),
                                 scale, w.cpu(), EPS, 0.3, p_round(decode, dtype, hq // hkv))
            assert_close(out[row:row + c], ref, tol, f"sequence {s}")
            row += c

    for s in (1, 2, 3):
        bm.add_sequence(s)
    step([1, 2, 3], [60, 17, 1])
    step([1, 2], [43, 30])
    bm.fork(1, 4)                        # 103 tokens: the last block is shared and part-filled
    for _ in range(3):
        step([1, 4, 2, 3], [1, 1, 1, 1])
    step([3, 4], [33, 2])


# A few query tiles, for half of the SMs at most, against long caches: clusters of 2, 3,
# 4, 6, 8 or 16 blocks share a tile's keys where the table holds two key tiles a block and
# all clusters run at once.
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dtype", [
    (4, 1, 128, "bf16"), (1, 1, 64, "f16"), (3, 1, 64, "bf16"), (5, 1, 128, "f16"),
    (14, 2, 128, "bf16"), (128, 1, 64, "f16"), (96, 1, 128, "bf16")])
@pytest.mark.parametrize("lens,chunks", [
    ([4100], [1]), ([2049, 4096, 130, 7], [1, 1, 1, 1]), ([3000, 257, 1], [9, 8, 1]),
    ([2700, 0, 640], [23, 0, 31])])
def test_prefill_shares_out_keys(pa, hq, hkv, d, dtype, norm, lens, chunks):
    x = Pool(lens, hq, hkv, d, dtype, chunks=chunks, norm=norm, seed=hq + d)
    x.check(x.prefill(pa))
    first = x.out.clone()
    x.prefill(pa, workspace=None)                            # neither order nor workspace matter
    assert torch.equal(x.out, first)


@pytest.mark.parametrize("hq,hkv,d", [(8, 4, 128), (4, 4, 64)])
@pytest.mark.parametrize("n", [5, 8, 11])                    # up to 6 blocks a tile
def test_prefill_shares_out_keys_of_several(pa, hq, hkv, d, n):
    lens = [1100 + 97 * i for i in range(n)]
    x = Pool(lens, hq, hkv, d, "bf16", chunks=[1 + 5 * i for i in range(n)], seed=n)
    x.check(x.prefill(pa))


@pytest.mark.parametrize("hq,hkv,d,dtype", [(2, 1, 128, "bf16"), (1, 1, 64, "f16")])
@pytest.mark.parametrize("n", [127, 128, 129, 1025, 2300])
def test_prefill_whole_prompt_shares_out_keys(pa, hq, hkv, d, dtype, n):
    x = Pool([n], hq, hkv, d, dtype, chunks=[n], seed=n, maxb=160)
    x.check(x.prefill(pa))


@pytest.mark.parametrize("n", [1, 127, 128, 255, 256, 257, 384, 511, 512, 513, 900, 1023, 1024, 1025])
def test_prefill_short_sequences_in_a_wide_table(pa, n):
    """How many of a cluster's blocks share a sequence's keys follows its length."""
    x = Pool([n, 2500, 33], 4, 1, 128, "f16", chunks=[min(n, 13), 2, 5], seed=n, maxb=400)
    x.check(x.prefill(pa))


def test_prefill_shared_out_large_scores(pa):
    x = Pool([4000, 2100], 4, 1, 128, "bf16", chunks=[20, 3], seed=3)
    x.scale = 4.0                                            # maxima grow from block to block
    x.check(x.prefill(pa))


def test_prefill_shared_out_reports(pa):
    x = Pool([2100, 2500, 2300], 4, 1, 64, "bf16", chunks=[4, 30, 2], seed=4)
    x.k.nan_to_num_(0.0)
    x.v.nan_to_num_(0.0)
    good = x.prefill(pa).clone()
    r0, pos = x.rows(1)
    keep = torch.ones(good.shape[0], dtype=torch.bool, device="cuda")
    keep[r0:r0 + len(pos)] = False
    x.tables[1, 100] = x.k.shape[0]
    out = x.prefill(pa).clone()
    assert pa.get_device_error() == pa.DEVERR["TABLE_RANGE"]
    assert torch.equal(out[keep], good[keep])
    x.tables.copy_(x.tables_h)
    for value in (-1, 16 * x.tables.shape[1] + 1):
        x.lens[1] = value
        out = x.prefill(pa).clone()
        assert pa.get_device_error() & pa.DEVERR["SEQLEN_RANGE"]
        assert torch.equal(out[keep], good[keep])


def test_prefill_shared_out_in_a_graph_and_on_two_streams(pa):
    xs = [Pool([3900, 33, 1400], 8, 2, 128, "bf16", chunks=[9, 9, 9], seed=30 + i)
          for i in range(2)]
    want = [x.prefill(pa, workspace=None).clone() for x in xs]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):                                      # at once
        for x, s in zip(xs, ss):
            x.prefill(pa, workspace=None, stream=s)
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        assert torch.equal(x.out[:w.shape[0]], w)            # bit-stable too
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            for x in xs:
                x.prefill(pa, workspace=None)
    for x in xs:
        x.out.fill_(7.0)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        assert torch.equal(x.out[:w.shape[0]], w)
        x.check(x.out[:w.shape[0]])


# Few runs, each cut into many pieces: merged by a block per run and head
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dtype", [
    (4, 1, 128, "bf16"), (1, 1, 64, "f16"), (7, 1, 128, "f16"), (16, 1, 64, "bf16"),
    (32, 2, 128, "bf16"), (10, 2, 64, "f16"), (8, 8, 64, "bf16")])
@pytest.mark.parametrize("lens", [[6000], [700], [130], [0, 2500, 17], [2049, 1, 300, 16]])
def test_decode_few_runs_of_many_pieces(pa, hq, hkv, d, dtype, norm, lens):
    x = Pool(lens, hq, hkv, d, dtype, norm=norm, seed=hq + d + len(lens), maxb=400)
    x.check(x.decode(pa))
    first = x.out.clone()
    x.decode(pa)
    assert torch.equal(x.out, first)


def test_decode_few_runs_large_scores(pa):
    x = Pool([5000], 4, 1, 128, "bf16", seed=3)
    x.scale = 4.0                                            # maxima differ from piece to piece
    x.check(x.decode(pa))


def test_decode_few_runs_in_a_graph_with_changing_lengths(pa):
    x = Pool([3000, 2000], 4, 1, 64, "f16", seed=5)
    x.decode(pa)
    g = torch.cuda.CUDAGraph()
    ws = pa.diff_decode_workspace_for(x.q, x.k, x.tables)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        x.decode(pa, workspace=ws)
        x.decode(pa, workspace=ws)
    for lens in ([3000, 2000], [5, 2000], [0, 33], [2999, 0], [1, 1]):
        x.lens_h = lens
        x.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        x.k.nan_to_num_(0.5)
        x.v.nan_to_num_(0.5)
        x.out.fill_(7.0)
        g.replay()
        x.check(x.out[:2])
    assert pa.get_device_error() == 0


# Grids of more blocks than SMs, which alone follow the work order
def ordered(pa, x, longest=None, by_seq=False, pairs=None):
    """A prefill of x that has to make a work order: the grid is large enough, and the
    order's head says how many (sequence, unit) pairs it holds and of which kind it is."""
    longest = max(x.chunks) if longest is None else longest
    n, (hq, hkv) = len(x.chunks), (x.q_h.shape[1], x.k_h.shape[1])
    tokens = 128 // (hq // hkv)                              # of a query tile
    tiles = 1 if longest <= tokens else 2                    # of a unit
    units = -(-longest // (tiles * tokens))
    props = torch.cuda.get_device_properties(0)
    assert units * tiles * n * hkv > props.multi_processor_count
    assert 2 * -(-longest // tokens) * n * hkv > props.multi_processor_count
    kv = sum(L for L, c in zip(x.lens_h, x.chunks) if c) * hkv * x.k_h.shape[3] * 4
    assert (kv > props.L2_cache_size) == by_seq
    ws = torch.full((pa.diff_prefill_workspace_size(n, longest, hq, hkv),), 0x5a,
                    dtype=torch.uint8, device="cuda")
    x.prefill(pa, longest=longest, workspace=ws)
    want = sum(min(units, -(-c // (tiles * tokens))) for c in x.chunks)
    assert ws[:8].view(torch.int32).tolist() == [want, int(by_seq)]
    return x.out[:x.start_h[-1]].clone()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dtype", [
    (10, 2, 128, "bf16"), (21, 3, 64, "f16"), (24, 8, 64, "bf16"), (8, 8, 128, "f16")])
def test_prefill_ordered(pa, hq, hkv, d, dtype, norm):
    lens = [1, 300, 140, 129, 0, 517, 40, 700]
    x = Pool(lens, hq, hkv, d, dtype, chunks=[1, 300, 3, 129, 0, 517, 0, 333], norm=norm, seed=hq)
    got = ordered(pa, x)
    x.check(got)
    assert torch.equal(x.prefill(pa, workspace=None), got)   # the order changes no result
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype", [(16, 4, 64, "f16"), (20, 4, 128, "bf16")])
def test_prefill_ordered_units_of_one_tile(pa, hq, hkv, d, dtype):
    rng = np.random.default_rng(9)
    chunks = [0, 25, 1] + rng.integers(0, 26, 45).tolist()
    lens = [c + int(rng.integers(0, 400)) for c in chunks]
    x = Pool(lens, hq, hkv, d, dtype, chunks=chunks, seed=40)
    got = ordered(pa, x)
    x.check(got)
    assert torch.equal(x.prefill(pa, workspace=None), got)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype,chunks", [
    (16, 8, 128, "bf16", [400, 130, 257]), (24, 8, 128, "f16", [260, 0, 85]),
    (32, 16, 64, "f16", [130, 70, 90])])
def test_prefill_ordered_by_sequence(pa, hq, hkv, d, dtype, chunks):
    # K/V past L2
    x = Pool([13500, 12001, 24500], hq, hkv, d, dtype, chunks=chunks, seed=15)
    got = ordered(pa, x, by_seq=True)
    x.check(got)
    assert torch.equal(x.prefill(pa, workspace=None), got)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype,longest,kept", [
    (16, 8, 128, "f16", 130, 128),                           # 3 units of 128 tokens, 2 in the grid
    (24, 8, 64, "bf16", 168, 168),                           # 4 units of 84, 2 in the grid
    (56, 8, 64, "f16", 18, 288)])                            # 17 units of 18, 1 in the grid
def test_prefill_ordered_longest_chunk_understated(pa, hq, hkv, d, dtype, longest, kept):
    chunks = [15, 300, 0, 1, 18] + [10] * 16
    x = Pool([90, 400, 0, 17, 18] + [33] * 16, hq, hkv, d, dtype, chunks=chunks, seed=8)
    good = ordered(pa, x)
    x.check(good)
    x.out.fill_(7.0)
    out = ordered(pa, x, longest=longest)
    assert pa.get_device_error() == pa.DEVERR["QUERY_RANGE"]
    skipped = slice(15, 15 + kept)
    assert bool((out[skipped] == 7).all())
    good[skipped] = 7
    assert torch.equal(out, good)


@pytest.mark.parametrize("n", [640, 768, 769, 895, 896, 1535, 1536, 1537, 2047, 2048, 2049])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (3, 1, 64)])
def test_prefill_shares_of_part_of_a_cluster(pa, n, hq, hkv, d):
    """A wide table gives a tile a cluster of 16 blocks; a sequence of 5 key tiles uses 2
    of them, of 6 and 7 three, of 12 to 15 six, of 16 and more eight."""
    x = Pool([n, 3000, 1], hq, hkv, d, "bf16", chunks=[7, 2, 1], seed=n, maxb=400)
    x.check(x.prefill(pa))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 64, "f16"), (8, 1, 128, "bf16"),
                                            (22, 2, 128, "f16"), (16, 1, 64, "bf16")])
def test_decode_shared_blocks(pa, hq, hkv, d, dtype):
    """Samples of one prompt: neighbours' tables name the same blocks, one names a block
    twice."""
    x = Pool([700, 700, 690, 33, 40, 1500], hq, hkv, d, dtype, seed=hq, maxb=100)
    for s, n in ((1, 43), (2, 43), (4, 2)):
        x.tables_h[s, :n] = x.tables_h[s - 1, :n]
    x.tables_h[5, 3] = x.tables_h[5, 4]
    x.tables.copy_(x.tables_h)
    x.check(x.decode(pa))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("kind,chunks", [("decode", None), ("prefill", [3, 40, 1]),
                                         ("prefill", [3, 400, 1])])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (12, 2, 64), (24, 2, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_queries_stay_apart(pa, kind, chunks, hq, hkv, d, bad):
    x = Pool([700, 1400, 33], hq, hkv, d, "bf16", chunks=chunks, seed=7)
    run = x.decode if kind == "decode" else x.prefill
    good = run(pa).clone()
    row = x.rows(1)[0]
    x.q[row, 1, 3] = bad                                     # one head's first map
    x.q[row, hq - 1, d - 1] = bad                            # another's second
    out = run(pa)
    assert not bool(torch.isfinite(out[row, [1, hq - 1]]).any())
    keep = torch.ones(good.shape[:2], dtype=torch.bool, device="cuda")
    keep[row, 1] = keep[row, hq - 1] = False
    assert torch.equal(out[keep], good[keep])


def test_prefill_ordered_on_two_streams_and_in_two_graphs(pa):
    xs = [Pool([700, 300, 128, 513, 64], 16, 8, 128, "bf16", chunks=[700, 299, 128, 1, 64],
               seed=50 + i) for i in range(2)]
    want = [ordered(pa, x) for x in xs]
    for x, w in zip(xs, want):
        x.check(w, only=[1, 3])
    ss = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s in zip(xs, ss):
            x.prefill(pa, stream=s)
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        assert torch.equal(x.out[:w.shape[0]], w)
        x.out.fill_(7.0)
    graphs = []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.prefill(pa)
    for _ in range(10):
        for g, s in zip(graphs, ss):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        assert torch.equal(x.out[:w.shape[0]], w)
    assert pa.get_device_error() == 0
