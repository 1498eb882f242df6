"""Block selection, decode over selected blocks, weight accounting and eviction on the
GPU against their definitions in 64 bits."""
import math

import pytest
import torch

import sparse_util as su

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
SCALE = {64: 0.125, 128: 0.088}


def gen(*key):
    return torch.Generator().manual_seed(hash(key) % (2 ** 31))


def cuda(*xs):
    return [x.cuda() if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32).cuda()
            for x in xs]


def check(pa, want=0):
    torch.cuda.synchronize()
    assert pa.get_device_error() == want


# ---------------------------------------------------------------------------
# block_bounds
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt,d,hkv", [("f16", 64, 1), ("bf16", 128, 8), ("f16", 128, 3),
                                      ("bf16", 64, 5)])
@pytest.mark.parametrize("which", ["all", "step", "chunk"])
def test_bounds(pa, dt, d, hkv, which):
    g = gen(1, d, hkv)
    lens = [0, 1, 15, 16, 17, 300, 33, 0, 129]
    tables, nb = su.tables_for(g, lens)
    k = su.pool(g, nb, hkv, d, DT[dt], su.dead_slots(tables, lens, nb))
    old = su.pool(g, nb, hkv, d, DT[dt])[:, :, :2].contiguous()
    starts = {"all": None, "step": [max(0, n - 1) for n in lens],
              "chunk": [n // 2 for n in lens]}[which]
    ref = su.bounds(old, k, tables, lens, starts)
    b, kk, tt, ll = cuda(old, k, tables, lens)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda()
    assert pa.block_bounds(b, kk, tt, ll, starts=st) is b
    check(pa)
    assert torch.equal(su.bits(b), su.bits(ref))


def test_bounds_of_odd_values(pa):
    g = gen(2)
    tables, nb = su.tables_for(g, [40])
    k = su.pool(g, nb, 2, 64, torch.bfloat16)
    blk = tables[0].long()
    k[blk[0], 0, 3, 5] = math.nan
    k[blk[0], 1, 15, 6] = math.inf
    k[blk[1], 0, 0, 7] = -math.inf
    k[blk[2], 1, 8, 9] = math.nan                      # past the end: not live
    b = torch.zeros(nb, 2, 2, 64, dtype=torch.bfloat16)
    ref = su.bounds(b, k, tables, [40])
    got = pa.block_bounds(*cuda(b, k, tables, [40])).cpu()
    check(pa)
    assert bool(torch.isnan(got[blk[0], 0, :, 5]).all())
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(ref.float()))


def test_bounds_of_many_sequences(pa):
    g = gen(3)
    lens = [int(x) for x in torch.randint(0, 50, (4500,), generator=g)]
    tables, nb = su.tables_for(g, lens)
    k = su.pool(g, nb, 2, 64, torch.float16)
    b = torch.zeros(nb, 2, 2, 64, dtype=torch.float16)
    got = pa.block_bounds(*cuda(b, k, tables, lens))
    check(pa)
    assert torch.equal(got.cpu(), su.bounds(b, k, tables, lens))


def test_bounds_report_bad_arguments(pa):
    g = gen(4)
    tables, nb = su.tables_for(g, [40, 40, 40])
    k = su.pool(g, nb, 2, 64, torch.float16)
    b = torch.zeros(nb, 2, 2, 64, dtype=torch.float16)
    bad = tables.clone()
    bad[1, 1], bad[2, 0] = nb, -5
    ref = b.clone()
    for i, j in ((0, 0), (0, 1), (0, 2), (1, 0), (1, 2), (2, 1), (2, 2)):
        t = int(tables[i, j])
        live = k[t, :, :16 if j < 2 else 8]
        ref[t, :, 0], ref[t, :, 1] = live.amin(1), live.amax(1)
    bb, kk, tt, ll = cuda(b, k, bad, [40, 40, 40])
    pa.block_bounds(bb, kk, tt, ll)
    check(pa, pa.DEVERR["TABLE_RANGE"])
    assert torch.equal(bb.cpu(), ref)
    pa.block_bounds(bb, kk, *cuda(tables, [40, 49, -1]))
    check(pa, pa.DEVERR["SEQLEN_RANGE"])
    bb.zero_()
    pa.block_bounds(bb, kk, *cuda(tables, [40, 40, 40], [-1, 41, 40]))
    check(pa, pa.DEVERR["QUERY_RANGE"])
    assert torch.equal(bb.cpu(), su.bounds(b, k, tables, [40, 0, 0]))


def test_bounds_after_a_step_of_a_padded_batch(pa):
    # starts = seq_lens - 1, also of sequences without tokens
    g = gen(72)
    lens = [0, 40, 0, 1, 16, 0]
    tables, nb = su.tables_for(g, lens)
    k = su.pool(g, nb, 3, 64, torch.bfloat16)
    old = su.pool(g, nb, 3, 64, torch.bfloat16)[:, :, :2].contiguous()
    b, kk, tt, ll = cuda(old, k, tables, lens)
    pa.block_bounds(b, kk, tt, ll, starts=ll - 1)
    check(pa)
    ref = su.bounds(old, k, tables, lens, [max(0, n - 1) for n in lens])
    assert torch.equal(su.bits(b), su.bits(ref))
    # other starts of empty sequences, and -1 of others, are none
    for i, x in ((0, -2), (0, 1), (1, -1)):
        starts = ll - 1
        starts[i] = x
        pa.block_bounds(b, kk, tt, ll, starts=starts)
        check(pa, pa.DEVERR["QUERY_RANGE"])


# ---------------------------------------------------------------------------
# select_blocks
# ---------------------------------------------------------------------------
def run_select(pa, q, b, tables, lens, keep, first, last, workspace=None):
    n, hkv = q.shape[0], b.shape[1]
    tiles = torch.full((n, hkv, keep), 77, dtype=torch.int32, device="cuda")
    held = torch.full((n, hkv), 77, dtype=torch.int32, device="cuda")
    pa.select_blocks(tiles, held, *cuda(q, b, tables, lens), keep_first=first, keep_last=last,
                     workspace=workspace)
    return tiles, held


def same_choice(pa, q, b, tables, lens, keep, first, last):
    got = run_select(pa, q, b, tables, lens, keep, first, last)
    check(pa)
    ref = su.select(q, b, tables, lens, keep, first, last)
    assert torch.equal(got[1].cpu(), ref[1])
    assert torch.equal(got[0].cpu(), ref[0])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d,hkv,g", [(64, 2, 1), (128, 2, 4), (128, 3, 5), (64, 1, 8),
                                     (128, 1, 9), (64, 2, 16), (128, 1, 16)])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 1), (7, 1, 2), (64, 4, 8), (5, 2, 3)])
def test_select(pa, dt, d, hkv, g, keep, first, last):
    r = gen(5, d, g, keep)
    lens = [0, 1, 16, 17, 112, 113, 900, 1024, 1025, 5000]
    tables, nb = su.tables_for(r, lens)
    k = su.pool(r, nb, hkv, d, DT[dt])
    b = su.bounds(torch.zeros(nb, hkv, 2, d, dtype=DT[dt]), k, tables, lens)
    q = torch.randn(len(lens), hkv * g, d, generator=r).to(DT[dt])
    same_choice(pa, q, b, tables, lens, keep, first, last)


def test_select_of_a_long_sequence(pa):
    r = gen(6)
    lens = [131072, 40000, 16]
    tables, nb = su.tables_for(r, lens)
    b = torch.randn(nb, 2, 2, 128, generator=r).to(torch.bfloat16).sort(2).values.contiguous()
    q = torch.randn(3, 8, 128, generator=r).to(torch.bfloat16)
    same_choice(pa, q, b, tables, lens, 256, 4, 8)
    same_choice(pa, q, b, tables, lens, 8191, 0, 1)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_select_between_close_scores(pa, dt):
    # one block's bounds, changed by a unit in the last place in one small channel each
    r = gen(7)
    n = 3000
    lens = [16 * n]
    tables, nb = su.tables_for(r, lens)
    b = torch.randn(1, 1, 2, 128, generator=r).sort(2).values.to(DT[dt]).repeat(nb, 1, 1, 1)
    c = torch.randint(0, 128, (nb,), generator=r)
    q = torch.randn(1, 4, 128, generator=r).to(DT[dt])
    at = torch.arange(nb)
    for side in range(2):
        raw = b.view(torch.int16)
        raw[at, 0, side, c] = raw[at, 0, side, c] ^ (torch.rand(nb, generator=r) < 0.5).short()
    for keep in (2, 40, 700, 2500):
        same_choice(pa, q, b, tables, lens, keep, 0, 1)
    # few of them close to the last one kept, the others far
    b[at[torch.rand(nb, generator=r) < 0.9]] *= 0.5
    for keep in (2, 40, 250):
        same_choice(pa, q, b, tables, lens, keep, 0, 1)


def test_select_between_equal_scores(pa):
    r = gen(8)
    lens = [16 * 2000, 16 * 100]
    tables, nb = su.tables_for(r, lens)
    q = torch.randn(2, 4, 64, generator=r).half()
    for b in (torch.zeros(nb, 2, 2, 64).half(),
              torch.randn(1, 2, 2, 64, generator=r).half().sort(2).values.repeat(nb, 1, 1, 1)):
        same_choice(pa, q, b, tables, lens, 50, 3, 2)
        same_choice(pa, q * 0, b, tables, lens, 1, 0, 1)
        b[tables[0, 1500].long()] *= 2
        b[tables[0, 7].long()] *= 2
        same_choice(pa, q, b, tables, lens, 50, 0, 1)


def test_select_with_infinities(pa):
    r = gen(9)
    lens = [16 * 300, 16 * 90]
    tables, nb = su.tables_for(r, lens)
    q = torch.randn(2, 8, 128, generator=r).bfloat16()
    b = torch.randn(nb, 2, 2, 128, generator=r).bfloat16().sort(2).values.contiguous()
    for j, x in ((5, math.inf), (40, -math.inf), (41, math.nan), (250, math.nan), (280, math.inf)):
        b[tables[0, j].long(), 0, j % 2, j % 128] = x
    b[tables[1].long(), 1, 0, 3] = math.nan                          # all of a head's
    for keep in (2, 4, 5, 6, 7, 40):
        same_choice(pa, q, b, tables, lens, keep, 0, 1)
    q[0, 1, 9] = math.inf
    same_choice(pa, q, b, tables, lens, 40, 1, 1)


def test_select_of_many_sequences(pa):
    r = gen(10)
    lens = [int(x) for x in torch.randint(0, 200, (2300,), generator=r)]
    tables, nb = su.tables_for(r, lens)
    b = torch.randn(nb, 1, 2, 64, generator=r).half().sort(2).values.contiguous()
    q = torch.randn(2300, 2, 64, generator=r).half()
    same_choice(pa, q, b, tables, lens, 5, 1, 1)


@pytest.mark.parametrize("runs,hkv", [(3, 1), (400, 1), (40, 8)])
def test_select_in_long_tables(pa, runs, hkv):
    # few runs: the scores apart; many: a block each
    r = gen(42, runs, hkv)
    lens = [int(x) for x in torch.randint(0, 16 * 300, (runs,), generator=r)]
    lens[1] = 16 * 300
    tables, nb = su.tables_for(r, lens)
    b = torch.randn(nb, hkv, 2, 64, generator=r).half().sort(2).values.contiguous()
    q = torch.randn(runs, hkv, 64, generator=r).half()
    same_choice(pa, q, b, tables, lens, 20, 1, 1)
    bad, as_zero = tables.clone(), tables.clone()
    bad[1, 299], bad[1, 7], as_zero[1, 299], as_zero[1, 7] = nb, -1, 0, 0
    got = run_select(pa, q, b, bad, lens, 20, 0, 1)
    check(pa, pa.DEVERR["TABLE_RANGE"])
    assert torch.equal(got[0].cpu(), su.select(q, b, as_zero, lens, 20, 0, 1)[0])


@pytest.mark.parametrize("runs", [2, 310])
def test_select_of_more_scores_than_fit(pa, runs):
    # a table wider than a thread block's shared memory holds scores for
    r = gen(43, runs)
    lens = [16 * (5 + i % 40) for i in range(runs)]
    lens[-1] = 16 * 16500
    tables, nb = su.tables_for(r, lens)
    b = torch.randn(nb, 1, 2, 64, generator=r).half().sort(2).values.contiguous()
    q = torch.randn(runs, 2, 64, generator=r).half()
    same_choice(pa, q, b, tables, lens, 300, 2, 2)
    b[tables[-1].long()] = b[0].clone()                # and all equal
    same_choice(pa, q, b, tables, lens, 30, 2, 2)


def test_select_between_equal_scores_of_many_runs(pa):
    r = gen(44)
    lens = [16 * 300] * 5 + [16 * (1 + i % 30) for i in range(310)]
    tables, nb = su.tables_for(r, lens)
    b = torch.randn(1, 1, 2, 64, generator=r).half().sort(2).values.repeat(nb, 1, 1, 1)
    q = torch.randn(len(lens), 2, 64, generator=r).half()
    same_choice(pa, q, b, tables, lens, 20, 1, 1)


def test_select_reports_bad_arguments(pa):
    r = gen(11)
    lens = [16 * 20, 16 * 20]
    tables, nb = su.tables_for(r, lens)
    b = torch.randn(nb, 2, 2, 64, generator=r).half().sort(2).values.contiguous()
    q = torch.randn(2, 4, 64, generator=r).half()
    bad, as_zero = tables.clone(), tables.clone()
    bad[0, 3], bad[1, 19], bad[1, 2] = nb, -1, 2 ** 31 - 1
    as_zero[0, 3], as_zero[1, 19], as_zero[1, 2] = 0, 0, 0
    got = run_select(pa, q, b, bad, lens, 6, 0, 1)
    check(pa, pa.DEVERR["TABLE_RANGE"])
    assert torch.equal(got[0].cpu(), su.select(q, b, as_zero, lens, 6, 0, 1)[0])
    got = run_select(pa, q, b, tables, [321, -7], 6, 0, 1)
    check(pa, pa.DEVERR["SEQLEN_RANGE"])
    assert torch.equal(got[0].cpu(), su.select(q, b, tables, [320, 0], 6, 0, 1)[0])


# ---------------------------------------------------------------------------
# sparse_decode
# ---------------------------------------------------------------------------
def random_tiles(r, n, hkv, keep, nb, held):
    tiles = torch.full((n, hkv, keep), -1, dtype=torch.int32)
    for i in range(n):
        for h in range(hkv):
            m = (int(held[i, h]) + 15) // 16
            tiles[i, h, :m] = (torch.randint(0, nb, (m,), generator=r) * hkv + h).int()
    return tiles


@pytest.mark.parametrize("dt,d,hkv,g,n,keep", [
    ("f16", 64, 2, 1, 3, 5), ("bf16", 128, 8, 4, 4, 40), ("f16", 128, 1, 7, 5, 100),
    ("bf16", 64, 3, 16, 2, 17), ("f16", 64, 8, 2, 300, 9), ("bf16", 128, 2, 9, 1, 300)])
def test_sparse_decode(pa, dt, d, hkv, g, n, keep):
    r = gen(12, n, keep)
    nb = 50
    k, v = (su.pool(r, nb, hkv, d, DT[dt]) for _ in range(2))
    held = torch.randint(0, 16 * keep + 1, (n, hkv), generator=r).int()
    held[0, 0], held[-1, -1] = 0, 16 * keep
    if hkv > 1:
        held[0, 1] = 1
    tiles = random_tiles(r, n, hkv, keep, nb, held)
    # what lies past a list's tokens is not looked at: a tile of NaN for every last one
    q = torch.randn(n, hkv * g, d, generator=r).to(DT[dt])
    ref, tol = su.sparse_decode(q, k, v, tiles, held, SCALE[d])
    out = torch.full_like(q, math.nan).cuda()
    qq, kk, vv, tt, hh = cuda(q, k, v, tiles, held)
    assert pa.sparse_decode(out, qq, kk, vv, tt, hh, SCALE[d]) is out
    check(pa)
    su.close(out, ref, tol)
    again = torch.empty_like(out)
    pa.sparse_decode(again, qq, kk, vv, tt, hh, SCALE[d])
    assert torch.equal(su.bits(again), su.bits(out))


def test_sparse_decode_past_the_end_holds_anything(pa):
    r = gen(13)
    k, v = (su.pool(r, 8, 2, 128, torch.bfloat16) for _ in range(2))
    held = torch.tensor([[35, 20]], dtype=torch.int32)
    tiles = torch.tensor([[[0, 4, 8, -1], [3, 7, 2 ** 30, 99]]], dtype=torch.int32)
    q = torch.randn(1, 8, 128, generator=r).bfloat16()
    ref, tol = su.sparse_decode(q, k, v, tiles, held, 0.088)
    k[4, 0, 3:], v[4, 0, 3:], k[3, 1, 4:], v[3, 1, 4:] = (math.nan, math.inf, math.inf, math.nan)
    out = pa.sparse_decode(torch.empty_like(q).cuda(), *cuda(q, k, v, tiles, held), 0.088)
    check(pa)
    su.close(out, ref, tol)


@pytest.mark.parametrize("dt,d,hkv,g,n,keep", [
    ("f16", 64, 2, 1, 3, 5), ("bf16", 128, 8, 4, 4, 40), ("f16", 128, 1, 7, 5, 100),
    ("bf16", 64, 3, 16, 2, 17), ("f16", 64, 8, 2, 300, 9), ("bf16", 128, 2, 9, 1, 300),
    ("bf16", 64, 1, 9, 3, 700), ("f16", 128, 2, 16, 2, 500), ("bf16", 128, 1, 8, 1, 2000)])
def test_sparse_decode_past_the_end_of_every_list(pa, dt, d, hkv, g, n, keep):
    # every run's last tile is its own, and holds NaN and infinities past the run's tokens; so
    # do the tiles that are named past it
    r = gen(73, n, keep)
    nb = 50
    last = (n * hkv + hkv - 1) // hkv                  # blocks of last tiles, behind the others
    k, v = (su.pool(r, nb + last + 1, hkv, d, DT[dt]) for _ in range(2))
    held = torch.randint(0, 16 * keep + 1, (n, hkv), generator=r).int()
    held[0, 0], held[-1, -1] = 1, 16 * keep - 7
    tiles = random_tiles(r, n, hkv, keep, nb, held)
    for i in range(n):
        for h in range(hkv):
            used = (int(held[i, h]) + 15) // 16
            tiles[i, h, used:] = (nb + last) * hkv + h
            if used:
                tiles[i, h, used - 1] = nb * hkv + i * hkv + h
    q = torch.randn(n, hkv * g, d, generator=r).to(DT[dt])
    ref, tol = su.sparse_decode(q, k, v, tiles, held, SCALE[d])
    kt, vt = (x.view(-1, 16, d) for x in (k, v))
    for i in range(n):
        for h in range(hkv):
            m = int(held[i, h])
            at = int(tiles[i, h, (m - 1) // 16]) if m else 0
            if m % 16:
                kt[at, m % 16:], vt[at, m % 16:] = ((math.nan, math.inf), (math.inf, math.nan),
                                                    (-math.inf, math.nan))[(i + h) % 3]
    k[nb + last], v[nb + last] = math.nan, math.nan
    out = pa.sparse_decode(torch.full_like(q, math.nan).cuda(), *cuda(q, k, v, tiles, held),
                           SCALE[d])
    check(pa)
    su.close(out, ref, tol)


def test_sparse_decode_names_a_tile_twice(pa):
    r = gen(14)
    k, v = (su.pool(r, 4, 1, 64, torch.float16) for _ in range(2))
    tiles, held = torch.tensor([[[2, 2, 1]]], dtype=torch.int32), torch.tensor([[48]])
    q = torch.randn(1, 1, 64, generator=r).half()
    ref, tol = su.sparse_decode(q, k, v, tiles, held, 0.125)
    out = pa.sparse_decode(torch.empty_like(q).cuda(), *cuda(q, k, v, tiles, held.int()), 0.125)
    check(pa)
    su.close(out, ref, tol)


@pytest.mark.parametrize("scale", [0.0, -0.11])
def test_sparse_decode_with_any_scale(pa, scale):
    r = gen(51)
    k, v = (su.pool(r, 90, 2, 128, torch.bfloat16) for _ in range(2))
    held = torch.tensor([[800, 1], [0, 77]], dtype=torch.int32)
    tiles = random_tiles(r, 2, 2, 50, 90, held)
    q = torch.randn(2, 6, 128, generator=r).bfloat16()
    ref, tol = su.sparse_decode(q, k, v, tiles, held, scale)
    out = pa.sparse_decode(torch.empty_like(q).cuda(), *cuda(q, k, v, tiles, held), scale)
    check(pa)
    su.close(out, ref, tol)


def test_sparse_decode_reports_bad_arguments(pa):
    r = gen(15)
    k, v = (su.pool(r, 4, 2, 64, torch.float16) for _ in range(2))
    q = torch.randn(1, 4, 64, generator=r).half()
    tiles = torch.tensor([[[0, 8, 4], [-1, 1, 3]]], dtype=torch.int32)
    as_zero = torch.tensor([[[0, 0, 4], [0, 1, 3]]], dtype=torch.int32)
    held = torch.tensor([[48, 30]], dtype=torch.int32)
    out = pa.sparse_decode(torch.empty_like(q).cuda(), *cuda(q, k, v, tiles, held), 0.125)
    check(pa, pa.DEVERR["TABLE_RANGE"])
    su.close(out, *su.sparse_decode(q, k, v, as_zero, held, 0.125))
    out = pa.sparse_decode(out, *cuda(q, k, v, as_zero, torch.tensor([[49, -2]]).int()), 0.125)
    check(pa, pa.DEVERR["SEQLEN_RANGE"])
    su.close(out, *su.sparse_decode(q, k, v, as_zero, torch.tensor([[48, 0]]), 0.125))


# ---------------------------------------------------------------------------
# decode_mass
# ---------------------------------------------------------------------------
def mass_case(pa, r, lens, dt, d, hkv, g, decay, mb=None, q_gain=2.0, scale=None):
    scale = SCALE[d] if scale is None else scale
    tables, nb = su.tables_for(r, lens, mb)
    k, v = (su.pool(r, nb, hkv, d, DT[dt], su.dead_slots(tables, lens, nb)) for _ in range(2))
    n = len(lens)
    q = (torch.randn(n, hkv * g, d, generator=r) * q_gain).to(DT[dt])
    mass = torch.rand(n, hkv, 16 * tables.shape[1], generator=r) * 5
    # old entries that are not to be read: the newest token's, and all with decay 0
    for i, m in enumerate(lens):
        if decay == 0.0:
            mass[i, :, :m] = math.nan
        elif m:
            mass[i, :, m - 1] = math.nan
        mass[i, :, m:] = math.nan
    ref = su.decode_mass(q, mass, k, v, tables, lens, scale, decay)
    out = torch.full_like(q, math.nan).cuda()
    qq, mm, kk, vv, tt, ll = cuda(q, mass, k, v, tables, lens)
    got = pa.decode_mass(out, mm, qq, kk, vv, tt, ll, scale, decay=decay)
    assert got[0] is out and got[1] is mm
    check(pa)
    su.close(out, ref[0], ref[1], "out")
    su.mass_close(mm, ref[2], ref[3], "mass")
    for i, m in enumerate(lens):                       # past the end nothing is written
        assert torch.equal(su.bits(mm[i, :, m:]), su.bits(mass[i, :, m:]))
        if m:
            assert bool(torch.isfinite(mm[i, :, :m]).all())
    plain = torch.empty_like(out)
    pa.decode(plain, qq, kk, vv, tt, ll, scale)
    # the plain decode's sums, but for few long runs, whose pieces are added in another order
    # (never in a table of less than 44 blocks, two for each of 22 pieces)
    if tables.shape[1] < 44:
        assert torch.equal(su.bits(plain), su.bits(out))
    else:
        su.close(plain, ref[0], ref[1], "plain")


@pytest.mark.parametrize("dt,d,hkv,g", [("f16", 64, 8, 1), ("bf16", 128, 2, 4), ("f16", 128, 1, 5),
                                        ("bf16", 64, 2, 8), ("f16", 64, 1, 9),
                                        ("bf16", 128, 2, 16), ("f16", 128, 3, 2)])
@pytest.mark.parametrize("decay", [1.0, 0.9, 0.0])
def test_decode_mass(pa, dt, d, hkv, g, decay):
    mass_case(pa, gen(16, d, g), [0, 1, 15, 16, 17, 100, 128, 129, 1000, 2], dt, d, hkv, g, decay)


@pytest.mark.parametrize("lens,mb", [([20000], None), ([3], 600), ([9000, 1, 0, 4000], None),
                                     ([100] * 20, 8), ([127, 128, 1], 8)])
def test_decode_mass_cut_and_whole(pa, lens, mb):
    mass_case(pa, gen(17, len(lens)), lens, "bf16", 128, 2, 4, 1.0, mb)


@pytest.mark.parametrize("dt,d,hkv,g", [("f16", 64, 1, 1), ("bf16", 64, 3, 7), ("f16", 128, 1, 16),
                                        ("bf16", 128, 2, 2)])
@pytest.mark.parametrize("lens", [[30000], [5000, 40, 0, 9000]])
def test_decode_mass_of_few_long_sequences(pa, dt, d, hkv, g, lens):
    mass_case(pa, gen(61, d, g), lens, dt, d, hkv, g, 0.9)


@pytest.mark.parametrize("dt,d,hkv,g,n,keep", [("bf16", 128, 1, 8, 1, 2000), ("f16", 64, 2, 3, 2, 900),
                                               ("bf16", 64, 1, 16, 3, 700),
                                               ("f16", 128, 4, 1, 2, 500)])
def test_sparse_decode_of_few_long_lists(pa, dt, d, hkv, g, n, keep):
    r = gen(62, keep)
    k, v = (su.pool(r, 300, hkv, d, DT[dt]) for _ in range(2))
    held = torch.randint(8 * keep, 16 * keep + 1, (n, hkv), generator=r).int()
    held[-1, -1] = 5 if n > 1 else held[-1, -1]
    tiles = random_tiles(r, n, hkv, keep, 300, held)
    q = torch.randn(n, hkv * g, d, generator=r).to(DT[dt])
    ref, tol = su.sparse_decode(q, k, v, tiles, held, SCALE[d])
    out = pa.sparse_decode(torch.empty_like(q).cuda(), *cuda(q, k, v, tiles, held), SCALE[d])
    check(pa)
    su.close(out, ref, tol)


def test_decode_mass_of_many_sequences(pa):
    r = gen(18)
    lens = [int(x) for x in torch.randint(0, 40, (2200,), generator=r)]
    mass_case(pa, r, lens, "f16", 64, 1, 2, 0.5)


def test_decode_mass_of_far_apart_scores(pa):
    # weights from one to far below the smallest float
    mass_case(pa, gen(19), [700, 33, 1], "bf16", 128, 2, 4, 1.0, q_gain=30.0)


@pytest.mark.parametrize("scale", [0.0, -0.11])
def test_decode_mass_with_any_scale(pa, scale):
    mass_case(pa, gen(50), [700, 0, 33, 1, 6000], "bf16", 128, 2, 4, 0.5, scale=scale)


def test_decode_mass_of_shared_blocks(pa):
    r = gen(20)
    lens = [40, 40, 35]
    tables, nb = su.tables_for(r, [40])
    tables = tables.repeat(3, 1)
    k, v = (su.pool(r, nb, 2, 64, torch.float16) for _ in range(2))
    q, mass = torch.randn(3, 4, 64, generator=r).half(), torch.zeros(3, 2, 48)
    ref = su.decode_mass(q, mass, k, v, tables, lens, 0.125, 1.0)
    out, m = pa.decode_mass(torch.empty_like(q).cuda(), *cuda(mass, q, k, v, tables, lens), 0.125)
    check(pa)
    su.close(out, *ref[:2])
    su.mass_close(m, *ref[2:])


@pytest.mark.parametrize("dt,d,hkv,g,n,most", [("bf16", 128, 2, 16, 70, 32), ("f16", 64, 1, 5, 350, 170),
                                               ("bf16", 64, 8, 4, 33, 32)])
def test_decode_mass_in_parts(pa, dt, d, hkv, g, n, most):
    # wide tables: the scores of so many sequences are taken four gigabytes at a time
    mb, r, scale = 65536, gen(71, n), SCALE[d]
    assert 2 ** 30 // (hkv * 16 * mb * (g + g % 2)) == most
    lens = [(97 * i) % 300 for i in range(n)]
    tables, nb = su.tables_for(r, lens)
    k, v = (su.pool(r, nb, hkv, d, DT[dt], su.dead_slots(tables, lens, nb)) for _ in range(2))
    q = (torch.randn(n, hkv * g, d, generator=r) * 2).to(DT[dt])
    used = 16 * tables.shape[1]
    mass = torch.rand(n, hkv, used, generator=r) * 5
    ref = su.decode_mass(q, mass, k, v, tables, lens, scale, 0.9)
    mm = torch.full((n, hkv, 16 * mb), 7.0, device="cuda")
    mm[..., :used] = mass.cuda()
    tt = torch.full((n, mb), -1, dtype=torch.int32, device="cuda")
    tt[:, :tables.shape[1]] = tables.cuda()
    qq, kk, vv, ll = cuda(q, k, v, lens)
    out = torch.full_like(qq, math.nan)
    pa.decode_mass(out, mm, qq, kk, vv, tt, ll, scale, decay=0.9)
    check(pa)
    su.close(out, *ref[:2], "out")
    su.mass_close(mm[..., :used], *ref[2:], "mass")
    assert bool((mm[..., used:] == 7.0).all())


def test_decode_mass_workspaces_are_bounded(pa):
    size = pa.decode_mass_workspace_size
    assert 0 < size(512, 32, 8, 128, 8192) < 2 ** 32 + 2 ** 27
    sizes = [size(n, 32, 8, 128, 8192) for n in range(1, 600)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[260]
    assert size(2, 16, 1, 64, 2 ** 24) > 2 ** 33         # one sequence alone may be more
    # what no call takes
    assert size(2, 17, 1, 64, 8) == 0 and size(2 ** 15, 2 ** 4, 2 ** 4, 64, 2 ** 12) == 0
    assert size(2 ** 30, 2 ** 20, 2 ** 20, 64, 8) == 0


# ---------------------------------------------------------------------------
# prefill_mass
# ---------------------------------------------------------------------------
def chunk_case(pa, r, lens, chunks, dt, d, hkv, g, decay, mb=None, longest=None, lead=0):
    tables, nb = su.tables_for(r, lens, mb)
    k = su.pool(r, nb, hkv, d, DT[dt], su.dead_slots(tables, lens, nb))
    start = [lead]
    for c in chunks:
        start.append(start[-1] + c)
    q = torch.randn(start[-1] + 2, hkv * g, d, generator=r).to(DT[dt])
    q[:lead] = q[start[-1]:] = math.nan                # rows that are no sequence's
    mass = torch.rand(len(lens), hkv, 16 * tables.shape[1], generator=r) * 5
    for i, (m, c) in enumerate(zip(lens, chunks)):
        mass[i, :, m - c:] = math.nan
        if decay == 0.0 and c:
            mass[i] = math.nan
    ref, tol = su.prefill_mass(q, mass, k, tables, lens, start, SCALE[d], decay)
    mm, qq, kk, tt, ll, ss = cuda(mass, q, k, tables, lens, start)
    got = pa.prefill_mass(mm, qq, kk, tt, ll, ss, longest or max(chunks), SCALE[d], decay=decay)
    assert got is mm
    check(pa)
    su.mass_close(mm, ref, tol)
    for i, (m, c) in enumerate(zip(lens, chunks)):
        keep = m if c else 0
        assert torch.equal(su.bits(mm[i, :, keep:]), su.bits(mass[i, :, keep:]))
        assert bool(torch.isfinite(mm[i, :, :keep]).all())
    m2 = cuda(mass)[0]
    pa.prefill_mass(m2, qq, kk, tt, ll, ss, longest or max(chunks), SCALE[d], decay=decay)
    assert torch.equal(su.bits(m2), su.bits(mm))


@pytest.mark.parametrize("dt,d,hkv,g", [("f16", 64, 2, 4), ("bf16", 128, 1, 1), ("f16", 128, 2, 5),
                                        ("bf16", 64, 1, 16), ("f16", 64, 3, 7),
                                        ("bf16", 128, 2, 8), ("f16", 128, 1, 128)])
@pytest.mark.parametrize("decay", [1.0, 0.0])
def test_prefill_mass(pa, dt, d, hkv, g, decay):
    chunk_case(pa, gen(21, d, g), [150, 70, 1, 130, 0, 300, 128], [5, 70, 1, 0, 0, 129, 128], dt, d,
               hkv, g, decay)


@pytest.mark.parametrize("dt,d,hkv,g", [("f16", 64, 2, 4), ("bf16", 128, 1, 1), ("f16", 128, 2, 5),
                                        ("bf16", 64, 1, 16), ("f16", 64, 3, 7),
                                        ("bf16", 128, 2, 3), ("f16", 128, 1, 128)])
@pytest.mark.parametrize("decay", [0.9, 0.0])
def test_prefill_mass_of_short_sequences(pa, dt, d, hkv, g, decay):
    # small tables, chunks of one row block and of several
    most = 131072 // (304 * g)
    chunk_case(pa, gen(40, d, g), [150, 300, 1, 16, 0, 47, 17], [min(most, 5), min(most, 70), 1, 16
                                                               if most >= 16 else 3, 0, 0, 1],
               dt, d, hkv, g, decay)
    chunk_case(pa, gen(41, d, g), [33, 8, 1], [min(33, most), min(8, most), 1], dt, d, hkv, g, decay)


@pytest.mark.parametrize("keys,rows,g", [
    (512, 16, 1), (512, 1, 16), (256, 2, 16), (128, 16, 4), (64, 128, 1), (48, 42, 4), (160, 12, 4),
    (16, 16, 16), (32, 2, 128), (160, 70, 4), (176, 17, 16), (80, 3, 128), (64, 60, 6), (64, 30, 12)])
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f16", 64)])
def test_prefill_mass_in_one_launch(pa, keys, rows, g, dt, d):
    # few products: the warps take rows, and parts of the keys where there are few rows
    rows = min(rows, keys)
    lens, chunks = [keys, keys - 3, 1, 0, rows, keys // 2 + 1], [rows, 1, 1, 0, rows, min(3, rows)]
    chunk_case(pa, gen(55, keys, rows, g), lens, chunks, dt, d, 2, g, 0.9, mb=keys // 16,
               longest=rows)


@pytest.mark.parametrize("c,g", [(1, 1), (1, 4), (2, 4), (3, 1), (1, 7), (5, 3), (4, 4), (2, 8),
                                 (1, 16), (16, 1), (3, 5)])
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("decay", [1.0, 0.0])
def test_prefill_mass_of_few_rows(pa, c, g, dt, d, decay):
    # chunks of at most 16 rows over keys that are read once
    lens = [3000, 0, 17, 640, 1, 5000, 33, 1024, 1025]
    chunks = [c, 0, min(c, 17), 1, 1, min(c, 2), 0, c, c]
    chunk_case(pa, gen(56, c, g), lens, chunks, dt, d, 3, g, decay, longest=c, lead=2)


def test_prefill_mass_of_few_rows_and_many_runs(pa):
    r = gen(57)
    lens = [int(x) for x in torch.randint(0, 700, (500,), generator=r)]
    lens[-3] = 900
    chunk_case(pa, r, lens, [min(n, 2) for n in lens], "bf16", 64, 2, 3, 0.9, longest=2)
    lens = [int(x) for x in torch.randint(0, 40, (2100,), generator=r)]
    lens[-3] = 800                                     # more sequences than the form takes
    chunk_case(pa, r, lens, [min(n, 2) for n in lens], "f16", 64, 1, 2, 0.9, longest=2)


def test_prefill_mass_with_the_workspace_of_longer_chunks(pa):
    r = gen(63)
    for n, length in ((2, 3000), (200, 90)):
        lens = [length - i % 50 for i in range(n)]
        tables, nb = su.tables_for(r, lens)
        k = su.pool(r, nb, 2, 64, torch.bfloat16)
        start = [2 * i for i in range(n + 1)]
        q = torch.randn(2 * n, 8, 64, generator=r).bfloat16()
        mass = torch.rand(n, 2, 16 * tables.shape[1], generator=r)
        ref, tol = su.prefill_mass(q, mass, k, tables, lens, start, 0.125, 1.0)
        qq, kk, tt, ll, ss = cuda(q, k, tables, lens, start)
        for longest in (2, 64, 500):
            ws = pa.prefill_mass_workspace_for(qq, kk, tt, longest)
            mm = mass.cuda()
            pa.prefill_mass(mm, qq, kk, tt, ll, ss, 2, 0.125, workspace=ws)
            check(pa)
            su.mass_close(mm, ref, tol)


def test_prefill_mass_of_few_rows_in_very_wide_tables(pa):
    # scores of all places of the tables would be more than a gigabyte: not kept
    chunk_case(pa, gen(59), [500, 40], [4, 4], "f16", 64, 3, 4, 1.0, mb=180000)
    chunk_case(pa, gen(60), [500, 40], [4, 4], "f16", 64, 3, 4, 1.0, mb=170000)


def test_prefill_mass_of_few_rows_reports_bad_arguments(pa):
    r = gen(58)
    lens = [1000, 1000]
    tables, nb = su.tables_for(r, lens)
    k = su.pool(r, nb, 1, 64, torch.float16)
    q = torch.randn(8, 4, 64, generator=r).half()
    old = torch.rand(2, 1, 1008, generator=r)
    kk, qq, tt = cuda(k, q, tables)

    def run(lens, start, longest, want, tables=tt):
        mm = old.cuda()
        pa.prefill_mass(mm, qq, kk, tables, *cuda(lens, start), longest, 0.125)
        check(pa, want)
        return mm.cpu()

    ref, bits = run(lens, [0, 2, 4], 2, 0), pa.DEVERR
    good, tol = su.prefill_mass(q, old, k, tables, lens, [0, 2, 4], 0.125, 1.0)
    su.mass_close(ref, good, tol)
    for a, b, e in (([1000, 1], [0, 2, 4], bits["QUERY_RANGE"]),
                    ([1000, 1009], [0, 2, 4], bits["SEQLEN_RANGE"]),
                    ([1000, -1], [0, 2, 4], bits["SEQLEN_RANGE"]),
                    (lens, [0, 2, 1], bits["QUERY_RANGE"]),
                    (lens, [0, 2, 9], bits["QUERY_RANGE"]),
                    (lens, [0, 2, 6], bits["QUERY_RANGE"])):
        got = run(a, b, 2, e)
        assert torch.equal(got[1], old[1]) and torch.equal(got[0], ref[0])
    bad, zero = tables.clone(), tables.clone()
    bad[1, 20], zero[1, 20] = nb, 0
    assert torch.equal(run(lens, [0, 2, 4], 2, bits["TABLE_RANGE"], bad.cuda()),
                       run(lens, [0, 2, 4], 2, 0, zero.cuda()))


@pytest.mark.parametrize("lens,chunks,g", [([5000], [64], 4), ([3000, 200], [700, 1], 2),
                                           ([1, 1], [1, 1], 4), ([2049], [2049], 1),
                                           ([9000, 130, 17], [1, 33, 17], 8)])
def test_prefill_mass_of_long_keys(pa, lens, chunks, g):
    chunk_case(pa, gen(22, g), lens, chunks, "bf16", 128, 1, g, 0.9)


@pytest.mark.parametrize("g,d,count", [(4, 128, 100), (3, 64, 77), (16, 64, 40), (1, 128, 60)])
def test_prefill_mass_of_many_units(pa, g, d, count):
    # shares of a few tiles that begin and end anywhere, units of one and of two query tiles
    r = gen(38, g)
    lens = [int(x) for x in torch.randint(0, 900, (count,), generator=r)]
    chunks = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 300, (count,), generator=r))]
    lens[3], chunks[3] = 900, 1
    chunk_case(pa, r, lens, chunks, "bf16", d, 2, g, 1.0)


def test_prefill_mass_of_many_sequences(pa):
    r = gen(52)
    for count, longest in ((700, 20), (2200, 150)):    # one row block, three
        lens = [int(x) for x in torch.randint(0, 60, (count,), generator=r)]
        chunks = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 20, (count,), generator=r))]
        lens[count - 2], chunks[count - 2] = 620, 20
        chunk_case(pa, r, lens, chunks, "f16", 64, 1, 4, 0.5, longest=longest, lead=3)


def test_prefill_mass_without_rows(pa):
    # a batch in which no sequence has any, then one that does, in every form
    r = gen(53)
    for mb, longest in ((60, 30), (60, 200), (8, 5)):
        lens = [16 * mb, 40, 0]
        tables, nb = su.tables_for(r, lens, mb)
        k = su.pool(r, nb, 2, 64, torch.float16)
        q = torch.randn(11, 4, 64, generator=r).half()
        old = torch.rand(3, 2, 16 * mb, generator=r)
        kk, qq, tt, ll, none, some = cuda(k, q, tables, lens, [4, 4, 4, 4], [1, 5, 11, 11])
        ref, tol = su.prefill_mass(q, old, k, tables, lens, [1, 5, 11, 11], 0.125, 1.0)
        for _ in range(10):
            mm = old.cuda()
            pa.prefill_mass(mm, qq, kk, tt, ll, none, longest, 0.125)
            kept = mm.clone()
            pa.prefill_mass(mm, qq, kk, tt, ll, none, longest, 0.125, decay=0.0)
            pa.prefill_mass(mm, qq, kk, tt, ll, some, longest if longest > 5 else 6, 0.125)
            assert torch.equal(kept.cpu(), old)
            su.mass_close(mm, ref, tol)
        check(pa)


def test_a_block_named_twice(pa):
    # by a table, in every call that reads
    r = gen(54)
    lens, hkv, d = [200, 90], 2, 64
    tables = torch.tensor([[3, 1, 3, 0, 2, 1, 3, 3, 4, 5, 0, 0, 2], [5, 5, 5, 5, 5, 1, 0, 0, 0, 0, 0,
                                                                   0, 0]], dtype=torch.int32)
    k, v = (su.pool(r, 6, hkv, d, torch.float16) for _ in range(2))
    q = torch.randn(2, 8, d, generator=r).half()
    mass = torch.rand(2, hkv, 208, generator=r)
    full = [208, 96]                                   # a block's bounds are of one length
    bnd = su.bounds(torch.zeros(6, hkv, 2, d, dtype=torch.float16), k, tables, full)
    got = pa.block_bounds(torch.zeros_like(bnd).cuda(), *cuda(k, tables, full))
    assert torch.equal(su.bits(got), su.bits(bnd))
    same_choice(pa, q, bnd, tables, lens, 5, 1, 1)
    ref = su.decode_mass(q, mass, k, v, tables, lens, 0.125, 1.0)
    out, m = pa.decode_mass(torch.empty_like(q).cuda(), *cuda(mass, q, k, v, tables, lens), 0.125)
    su.close(out, *ref[:2])
    su.mass_close(m, *ref[2:])
    for longest in (1, 300):                           # both forms
        ref, tol = su.prefill_mass(q, mass, k, tables, lens, [0, 1, 2], 0.125, 1.0)
        m = cuda(mass)[0]
        pa.prefill_mass(m, *cuda(q, k, tables, lens, [0, 1, 2]), longest, 0.125)
        su.mass_close(m, ref, tol)
    check(pa)


def test_prefill_mass_again_and_again(pa):
    r = gen(39)
    for count, most, c in ((1, 20000, 200), (5, 3000, 64), (20, 700, 33), (300, 100, 20)):
        lens = [int(x) for x in torch.randint(1, most, (count,), generator=r)]
        chunks = [min(n, c + i % 40) for i, n in enumerate(lens)]
        tables, nb = su.tables_for(r, lens)
        start = [0]
        for x in chunks:
            start.append(start[-1] + x)
        k, q = (torch.randn(s, generator=r).bfloat16().cuda()
                for s in ((nb, 2, 16, 128), (start[-1], 8, 128)))
        tt, ll, ss = cuda(tables, lens, start)
        first = None
        for _ in range(60):
            m = torch.zeros(count, 2, 16 * tables.shape[1], device="cuda")
            pa.prefill_mass(m, q, k, tt, ll, ss, max(chunks), 0.088)
            first = m if first is None else first
            assert torch.equal(m, first)
        check(pa)
        # every row gives a weight of one
        total = first.double().sum(-1).cpu()
        want = torch.tensor(chunks).double()[:, None] * 4
        assert bool(((total - want).abs() <= 2e-4 * want).all())


def test_prefill_mass_in_a_wide_table(pa):
    chunk_case(pa, gen(23), [300, 10], [20, 10], "f16", 64, 2, 4, 1.0, mb=500, longest=900)


def test_prefill_mass_chunk_by_chunk(pa):
    # a prompt in three chunks gives the weights of the prompt in one
    r = gen(24)
    tables, nb = su.tables_for(r, [200])
    k = su.pool(r, nb, 2, 64, torch.float16)
    q = torch.randn(200, 4, 64, generator=r).half()
    mm, kk, tt = cuda(torch.full((1, 2, 208), math.nan), k, tables)
    for a, b in ((0, 50), (50, 51), (51, 200)):
        pa.prefill_mass(mm, q[a:b].contiguous().cuda(), kk, tt, *cuda([b], [0, b - a]), b - a, 0.125)
    check(pa)
    ref, tol = su.prefill_mass(q, torch.zeros(1, 2, 208), k, tables, [200], [0, 200], 0.125, 1.0)
    su.mass_close(mm[..., :200], ref[..., :200], tol[..., :200])


def test_prefill_mass_reports_bad_arguments(pa):
    r = gen(25)
    lens = [100, 100]
    tables, nb = su.tables_for(r, lens)
    k = su.pool(r, nb, 1, 64, torch.float16)
    q = torch.randn(80, 4, 64, generator=r).half()
    old = torch.rand(2, 1, 112, generator=r)
    kk, qq, tt = cuda(k, q, tables)

    def run(lens, start, longest, want, tables=tt):
        mm = old.cuda()
        pa.prefill_mass(mm, qq, kk, tables, *cuda(lens, start), longest, 0.125)
        check(pa, want)
        return mm.cpu()

    good, _ = su.prefill_mass(q, old, k, tables, lens, [0, 40, 80], 0.125, 1.0)
    bits = pa.DEVERR
    ref = run(lens, [0, 40, 80], 40, 0)
    for a, b, c, e in (([100, 30], [0, 40, 80], 40, bits["QUERY_RANGE"]),
                       ([100, 113], [0, 40, 80], 40, bits["SEQLEN_RANGE"]),
                       ([100, -1], [0, 40, 80], 40, bits["SEQLEN_RANGE"]),
                       ([100, 100], [0, 40, 30], 40, bits["QUERY_RANGE"]),
                       ([100, 100], [0, 40, 90], 60, bits["QUERY_RANGE"]),
                       ([100, 100], [0, 40, 2 ** 31 - 1], 60, bits["QUERY_RANGE"])):
        got = run(a, b, c, e)
        assert torch.equal(got[1], old[1]) and torch.equal(got[0], ref[0])
    # a chunk beyond the last row block of the longest: 64 tokens of four heads
    got = run(lens, [0, 10, 80], 60, bits["QUERY_RANGE"])
    assert torch.equal(got[1], old[1])
    bad, zero = tables.clone(), tables.clone()
    bad[1, 2], zero[1, 2] = nb, 0
    assert torch.equal(run(lens, [0, 40, 80], 40, bits["TABLE_RANGE"], bad.cuda()),
                       run(lens, [0, 40, 80], 40, 0, zero.cuda()))


@pytest.mark.parametrize("lens,chunks,g,d,hkv,parts", [
    ([300, 70, 900, 40], [150, 70, 5, 0], 128, 64, 1, 3),
    ([700, 611, 65, 130], [600, 90, 65, 129], 16, 128, 2, 3),
    ([90, 17, 1, 64], [85, 17, 1, 64], 128, 128, 1, 2)])
@pytest.mark.parametrize("decay", [0.9, 0.0])
def test_prefill_mass_in_parts(pa, lens, chunks, g, d, hkv, parts, decay):
    # wide tables: the sums of so many row blocks are taken a gigabyte at a time
    mb = 65536
    tokens = 2 * (128 // g)
    blocks = (max(chunks) + tokens - 1) // tokens
    most = 2 ** 28 // (2 * len(lens) * hkv * 16 * mb)
    assert (blocks + most - 1) // most == parts
    chunk_case(pa, gen(70, g, d), lens, chunks, "bf16", d, hkv, g, decay, mb=mb)


@pytest.mark.parametrize("g,d", [(4, 64), (16, 128)])
def test_prefill_mass_with_a_far_bound_on_chunks(pa, g, d):
    # no chunk is longer than the tables: a bound above that asks for nothing more
    lens, chunks = [300, 960, 40, 0], [70, 500, 40, 0]
    size = pa.prefill_mass_workspace_size
    for hkv in (1, 3):
        full = size(4, 960, hkv * g, hkv, 60)
        assert 0 < full == size(4, 2000, hkv * g, hkv, 60) == size(4, 2 ** 31 - 1, hkv * g, hkv, 60)
    chunk_case(pa, gen(75, g), lens, chunks, "f16", d, 2, g, 0.9, mb=60, longest=10 ** 6)


def test_prefill_mass_workspaces_are_bounded(pa):
    size = pa.prefill_mass_workspace_size
    # a whole prompt of 131072 tokens, and 8 chunks of 8192 in tables for 32768
    for shape in ((1, 131072, 32, 8, 8192), (8, 8192, 32, 8, 2048)):
        assert 0 < size(*shape) < 2 ** 30 + 2 ** 25
    # that of longer chunks is no smaller
    sizes = [size(4, c, 32, 8, 8192) for c in range(1, 3000, 7)]
    assert sizes[1:] == sorted(sizes[1:]) and max(sizes) < 2 ** 30 + 2 ** 25
    # one row block alone may be more
    assert size(64, 65, 32, 8, 65536) > 2 ** 32
    # what no call takes
    assert size(2 ** 30, 8, 2 ** 21, 2 ** 20, 2 ** 10) == 0
    assert size(2 ** 15, 8, 2 ** 4, 2 ** 4, 2 ** 12) == 0


# ---------------------------------------------------------------------------
# evict
# ---------------------------------------------------------------------------
def evict_case(pa, r, lens, new_lens, first, last, dt="f16", d=64, hkv=2, mass=None, mb=None):
    tables, nb = su.tables_for(r, lens, mb)
    k, v = (su.pool(r, nb, hkv, d, DT[dt], su.dead_slots(tables, lens, nb)) for _ in range(2))
    if mass is None:
        mass = torch.randn(len(lens), hkv, 16 * tables.shape[1], generator=r).exp()
        for i, m in enumerate(lens):
            mass[i, :, m:] = math.nan
    elif callable(mass):
        mass = mass(len(lens), hkv, 16 * tables.shape[1])
    ref = su.evict(k, v, mass, tables, lens, new_lens, first, last)
    kk, vv, mm, tt, ll, nn = cuda(k, v, mass, tables, lens, new_lens)
    pa.evict(kk, vv, mm, tt, ll, nn, keep_first=first, keep_last=last)
    check(pa)
    for got, want in zip((mm, kk, vv), (ref[2], ref[0], ref[1])):
        assert torch.equal(su.bits(got), su.bits(want))


@pytest.mark.parametrize("dt,d,hkv", [("f16", 64, 2), ("bf16", 128, 3)])
@pytest.mark.parametrize("first,last", [(0, 0), (4, 32), (3, 0), (0, 5), (1, 300), (500, 7)])
def test_evict(pa, dt, d, hkv, first, last):
    evict_case(pa, gen(26, d, first), [0, 1, 2, 40, 40, 41, 100, 700, 257, 300, 33],
               [0, 0, 1, 40, 39, 16, 100, 64, 256, 0, 90], first, last, dt, d, hkv)


@pytest.mark.parametrize("lens,new,first,last", [
    ([20000], [2000], 4, 64), ([9000, 30000], [8999, 1], 0, 1), ([8192, 8193], [4096, 8000], 0, 128),
    ([40000], [39000], 10, 2000), ([1040] * 5, [1024] * 5, 4, 32), ([12000], [11000], 0, 11000)])
def test_evict_long(pa, lens, new, first, last):
    evict_case(pa, gen(27, len(lens), first), lens, new, first, last, "bf16", 128, 1)


def test_evict_in_wide_tables(pa):
    # more table entries than a block holds, and (many runs, a block each) more masses
    evict_case(pa, gen(45), [131200, 500], [100000, 40], 4, 64, "f16", 64, 1)
    lens = [3 + i % 50 for i in range(320)]
    lens[7], lens[200] = 40000, 35000
    evict_case(pa, gen(46), lens, [min(n, 20) if n < 100 else 1000 for n in lens], 4, 5, "f16", 64, 1)
    evict_case(pa, gen(47), lens, [min(n, 20) if n < 100 else 33000 for n in lens], 0, 40, "f16", 64,
               1, mass=lambda *x: torch.randint(0, 3, x, generator=gen(48)).float())


@pytest.mark.parametrize("runs,width", [(1, 4096), (30, 4096), (80, 8192), (150, 4096), (400, 2064),
                                        (400, 2048)])
def test_evict_by_blocks_and_clusters(pa, runs, width):
    # as many thread blocks to a run as the runs leave room for, from eight to one
    r = gen(49, runs)
    lens = [int(x) for x in torch.randint(0, 900, (runs,), generator=r)]
    lens[0] = width
    evict_case(pa, r, lens, [n // 2 for n in lens], 3, 20, "bf16", 64, 1, mb=width // 16)


def test_evict_ties_and_odd_masses(pa):
    lens, new = [500, 500, 333, 9100], [100, 499, 64, 5000]
    evict_case(pa, gen(28), lens, new, 2, 9, mass=lambda *s: torch.zeros(s))
    evict_case(pa, gen(29), lens, new, 2, 9,
               mass=lambda *s: torch.randint(0, 3, s, generator=gen(30)).float() - 1)

    def odd(*s):
        m = torch.randn(s, generator=gen(31))
        pick = torch.randint(0, 12, s, generator=gen(32))
        for i, x in enumerate((math.nan, math.inf, -math.inf, -0.0, 0.0, -math.nan)):
            m[pick == i] = x
        return m
    evict_case(pa, gen(33), lens, new, 2, 9, mass=odd)


def test_evict_of_many_sequences(pa):
    r = gen(34)
    lens = [int(x) for x in torch.randint(0, 60, (1500,), generator=r)]
    new = [int(x) for x in torch.randint(0, 60, (1500,), generator=r)]
    evict_case(pa, r, lens, new, 1, 4)


def test_evict_leaves_bad_sequences(pa):
    r = gen(35)
    lens = [100, 100, 100, 100]
    tables, nb = su.tables_for(r, lens)
    k, v = (su.pool(r, nb, 1, 64, torch.float16) for _ in range(2))
    mass = torch.rand(4, 1, 112, generator=r)
    bad = tables.clone()
    bad[2, 6] = nb
    for a, b, t, e in (([100, 113, 100, 100], [50] * 4, tables, "SEQLEN_RANGE"),
                       ([100, -1, 100, 100], [50] * 4, tables, "SEQLEN_RANGE"),
                       (lens, [50, -1, 50, 50], tables, "SEQLEN_RANGE"),
                       (lens, [50] * 4, bad, "TABLE_RANGE")):
        skip = 2 if t is bad else 1
        want = [100 if i == skip else 50 for i in range(4)]
        ref = su.evict(k, v, mass, tables, lens, want, 2, 10)
        kk, vv, mm, tt, ll, nn = cuda(k, v, mass, t, a, b)
        pa.evict(kk, vv, mm, tt, ll, nn, keep_first=2, keep_last=10)
        check(pa, pa.DEVERR[e])
        for got, x in zip((kk, vv, mm), ref):
            assert torch.equal(su.bits(got), su.bits(x))


# ---------------------------------------------------------------------------
# together, and on other streams
# ---------------------------------------------------------------------------
def test_a_prompt_is_cut_and_decoded_on(pa):
    """A prompt's weights, eviction, bounds, selection and a sparse decode, then decode
    steps that keep account, evict a block's worth and select again."""
    r = gen(36)
    hq, hkv, d, scale, keep, budget = 8, 2, 64, 0.125, 6, 160
    lens, mb = [300, 220], 24
    nb = 60
    tables = torch.randperm(nb, generator=r)[:2 * mb].reshape(2, mb).int()
    k, v = (su.pool(r, nb, hkv, d, torch.float16) for _ in range(2))
    mass = torch.full((2, hkv, 16 * mb), math.nan)
    bnd = torch.zeros(nb, hkv, 2, d, dtype=torch.float16)
    kk, vv, mm, bb, tt = cuda(k, v, mass, bnd, tables)
    q = torch.randn(64, hq, d, generator=r).half()
    pa.prefill_mass(mm, q.cuda(), kk, tt, *cuda(lens, [0, 32, 64]), 32, scale, decay=0.0)
    ref, tol = su.prefill_mass(q, mass, k, tables, lens, [0, 32, 64], scale, 0.0)
    su.mass_close(mm, ref, tol, "prompt")

    def cut(lens, new):
        nonlocal k, v
        before = mm.cpu()
        k, v, m = su.evict(kk.cpu(), vv.cpu(), before, tables, lens, new, 4, 16)
        pa.evict(kk, vv, mm, tt, *cuda(lens, new), keep_first=4, keep_last=16)
        for got, x in zip((kk, vv, mm), (k, v, m)):
            assert torch.equal(su.bits(got), su.bits(x))
        pa.block_bounds(bb, kk, tt, *cuda(new))
        return list(new)

    lens = cut(lens, [budget, budget])
    for step in range(17):
        lens = [n + 1 for n in lens]
        kn, vn = (torch.randn(2, hkv, d, generator=r).half() for _ in range(2))
        slots = torch.tensor([int(tables[i, (n - 1) // 16]) * 16 + (n - 1) % 16
                              for i, n in enumerate(lens)]).cuda()
        pa.reshape_and_cache(kn.cuda(), vn.cuda(), kk, vv, slots)
        q = torch.randn(2, hq, d, generator=r).half()
        before, k, v = mm.cpu(), kk.cpu(), vv.cpu()
        ll = torch.tensor(lens, dtype=torch.int32).cuda()
        pa.block_bounds(bb, kk, tt, ll, starts=ll - 1)
        if step % 2:
            out, _ = pa.decode_mass(torch.empty_like(q).cuda(), mm, *cuda(q, k, v), tt, ll, scale)
            ref = su.decode_mass(q, before, k, v, tables, lens, scale, 1.0)
            su.close(out, *ref[:2], "step")
            su.mass_close(mm, *ref[2:], "step")
        else:
            tiles, held = run_select(pa, q, bb.cpu(), tables, lens, keep, 1, 1)
            ref = su.select(q, su.bounds(bnd, k, tables, lens), tables, lens, keep, 1, 1)
            assert torch.equal(tiles.cpu(), ref[0]) and torch.equal(held.cpu(), ref[1])
            out = pa.sparse_decode(torch.empty_like(q).cuda(), q.cuda(), kk, vv, tiles, held, scale)
            su.close(out, *su.sparse_decode(q, k, v, *ref, scale), "step")
        if lens[0] % 16 == 0:
            lens = cut(lens, [n - 16 for n in lens])
    check(pa)


def test_a_batch_goes_on_after_an_eviction(pa):
    """The documented lines: sequences longer than new_lens are cut, the shorter one stays, each
    gets a token and a step counts it; then the batch changes its rows and its tables' width."""
    r = gen(74)
    hq, hkv, d, scale = 8, 2, 64, 0.125
    lens, nb, mb = [300, 40, 0, 100], 60, 20
    tables = torch.full((4, mb), -1, dtype=torch.int32)
    order = torch.randperm(nb, generator=r).int()
    tables[0, :19], tables[1, :3], tables[2, :1], tables[3, :7] = (order[:19], order[19:22],
                                                                   order[22:23], order[23:30])
    k, v = (su.pool(r, nb, hkv, d, torch.float16) for _ in range(2))
    mass = torch.full((4, hkv, 16 * mb), math.nan)
    kk, vv, mm, tt, ll, new = cuda(k, v, mass, tables, lens, [100] * 4)
    start = [0, 8, 12, 12, 20]
    q = torch.randn(20, hq, d, generator=r).half()
    pa.prefill_mass(mm, q.cuda(), kk, tt, ll, cuda(start)[0], 8, scale, decay=0.0)
    su.mass_close(mm, *su.prefill_mass(q, mass, k, tables, lens, start, scale, 0.0))
    before = mm.cpu()
    pa.evict(kk, vv, mm, tt, ll, new, keep_first=4, keep_last=16)
    ref = su.evict(k, v, before, tables, lens, [100] * 4, 4, 16)
    assert all(torch.equal(su.bits(x), su.bits(y)) for x, y in zip((kk, vv, mm), ref))
    ll = torch.minimum(ll, new)
    for step in range(3):
        where = tt.gather(1, (ll // 16).long()[:, None])[:, 0]
        kn, vn, q = (torch.randn(4, x, d, generator=r).half() for x in (hkv, hkv, hq))
        pa.reshape_and_cache(kn.cuda(), vn.cuda(), kk, vv, where.long() * 16 + ll % 16)
        ll += 1
        before = mm.cpu()
        out, _ = pa.decode_mass(torch.empty_like(q).cuda(), mm, q.cuda(), kk, vv, tt, ll, scale)
        ref = su.decode_mass(q, before, kk.cpu(), vv.cpu(), tt.cpu(), ll.tolist(), scale, 1.0)
        su.close(out, *ref[:2])
        su.mass_close(mm, *ref[2:])
        if step == 0:                                  # other rows, wider tables
            rows = torch.tensor([3, 0, 2, 1]).cuda()
            wide = torch.full((4, hkv, 16 * (mb + 5)), math.nan, device="cuda")
            wide[..., :16 * mb] = mm[rows]
            mm, ll = wide, ll[rows].contiguous()
            tt = torch.nn.functional.pad(tt[rows], (0, 5), value=-1).contiguous()
    assert ll.tolist() == [103, 103, 3, 43]
    check(pa)


class Step:
    """The six calls on state of their own, with workspaces of their own."""

    def __init__(self, pa, seed):
        r = gen(37, seed)
        self.pa, self.lens = pa, [700, 90, 0, 33]
        tables, nb = su.tables_for(r, self.lens)
        hkv, d = 2, 128
        self.k0, self.v0 = (su.pool(r, nb, hkv, d, torch.bfloat16) for _ in range(2))
        self.q0 = torch.randn(4, 8, d, generator=r).bfloat16()
        self.m0 = torch.rand(4, hkv, 16 * tables.shape[1], generator=r)
        (self.k, self.v, self.q, self.m, self.t, self.ll, self.new, self.start) = cuda(
            self.k0, self.v0, self.q0, self.m0, tables, self.lens, [300, 40, 0, 50],
            [0, 2, 3, 3, 4])
        self.b = torch.zeros(nb, hkv, 2, d, dtype=torch.bfloat16, device="cuda")
        self.tiles = torch.zeros(4, hkv, 6, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(4, hkv, dtype=torch.int32, device="cuda")
        self.out, self.out2 = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.ws = [pa.select_blocks_workspace_for(self.q, self.b, self.t),
                   pa.sparse_decode_workspace_for(self.q, self.k, self.tiles),
                   pa.decode_mass_workspace_for(self.q, self.k, self.t),
                   pa.prefill_mass_workspace_for(self.q, self.k, self.t, 2),
                   pa.evict_workspace_for(self.k, self.t)]

    def reset(self):
        for x, y in ((self.k, self.k0), (self.v, self.v0), (self.m, self.m0)):
            x.copy_(y)
        for x in (self.b, self.tiles, self.held, self.out, self.out2, *self.ws):
            x.zero_()
        torch.cuda.synchronize()

    def run(self, stream=None):
        pa = self.pa
        pa.block_bounds(self.b, self.k, self.t, self.ll, stream=stream)
        pa.select_blocks(self.tiles, self.held, self.q, self.b, self.t, self.ll, 1, 1, self.ws[0],
                         stream=stream)
        pa.sparse_decode(self.out, self.q, self.k, self.v, self.tiles, self.held, 0.088, self.ws[1],
                         stream=stream)
        pa.prefill_mass(self.m, self.q, self.k, self.t, self.ll, self.start, 2, 0.088,
                        workspace=self.ws[3], stream=stream)
        pa.decode_mass(self.out2, self.m, self.q, self.k, self.v, self.t, self.ll, 0.088, 0.9,
                       self.ws[2], stream=stream)
        pa.evict(self.k, self.v, self.m, self.t, self.ll, self.new, 2, 16, self.ws[4],
                 stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.b, self.tiles, self.held, self.out, self.out2, self.m,
                                    self.k, self.v)]


def same(a, b):
    return all(torch.equal(su.bits(x) if x.is_floating_point() else x.cpu(),
                           su.bits(y) if y.is_floating_point() else y.cpu()) for x, y in zip(a, b))


def test_streams_and_graphs(pa):
    a, b = Step(pa, 1), Step(pa, 2)
    want = []
    for x in (a, b):
        x.reset()
        x.run()
        want.append(x.results())
    # two at once on streams of their own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.reset(), b.reset()
        a.run(s1), b.run(s2)
        assert same(a.results(), want[0]) and same(b.results(), want[1])
    # captured, replayed together and again
    graphs = []
    for x, s in ((a, s1), (b, s2)):
        x.reset()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            x.run()
        graphs.append(gr)
    for _ in range(3):
        a.reset(), b.reset()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        assert same(a.results(), want[0]) and same(b.results(), want[1])
    check(pa)


def test_no_workspace_given(pa):
    a = Step(pa, 3)
    a.reset()
    a.run()
    want = a.results()
    a.reset()
    a.ws = [None] * 5
    a.run(torch.cuda.Stream())
    got = a.results()
    assert same(got, want)
    with pytest.raises(pa.PagedAttnError):
        pa.evict(a.k, a.v, a.m, a.t, a.ll, a.new,
                 workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))


def test_empty_batch(pa):
    z = torch.zeros(0, 4, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.float16, device="cuda")
    t = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    ll = torch.zeros(0, dtype=torch.int32, device="cuda")
    m = torch.zeros(0, 2, 48, device="cuda")
    tiles = torch.zeros(0, 2, 2, dtype=torch.int32, device="cuda")
    held = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    b = torch.zeros(3, 2, 2, 64, dtype=torch.float16, device="cuda")
    pa.block_bounds(b, k, t, ll)
    pa.select_blocks(tiles, held, z, b, t, ll)
    pa.sparse_decode(z.clone(), z, k, k, tiles, held, 1.0)
    pa.decode_mass(z.clone(), m, z, k, k, t, ll, 1.0)
    pa.prefill_mass(m, z, k, t, ll, torch.zeros(1, dtype=torch.int32, device="cuda"), 0, 1.0)
    pa.evict(k, k, m, t, ll, ll)
    check(pa)
