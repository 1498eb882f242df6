"""The block-selection, weight-accounting and eviction entry points refuse what they
cannot do, on the host, and their references are what the formulas say (no GPU)."""
import math

import pytest
import torch

import sparse_util as su

FAKE, OTHER = 0x1000, 0x2000
NAMES = ["pa_block_bounds", "pa_select_blocks", "pa_sparse_decode", "pa_decode_mass",
         "pa_prefill_mass", "pa_evict"]


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_260_gb300 import _build
    import paged_kv_cache_260_gb300 as pa
    _build.build()
    return pa.load()


def _call(lib, name, size=None, **kw):
    from paged_kv_cache_260_gb300 import _SPARSE_ARGS
    a = dict(out=OTHER, mass=FAKE, q=FAKE, k=FAKE, v=FAKE, bounds=FAKE, tables=FAKE, lens=FAKE,
             start=FAKE, starts=FAKE, new_lens=FAKE, tiles=FAKE, tile_lens=FAKE, ws=0, stream=0,
             wb=0, scale=0.1, decay=1.0, n=4, rows=32, longest=8, hq=8, hkv=2, d=128, bs=16, mb=8,
             nb=64, keep=4, first=1, last=1, dtype=0, reserved=0)
    assert not set(kw) - set(a)
    a.update(kw)
    return getattr(lib, name)(_SPARSE_ARGS.pack(_SPARSE_ARGS.size if size is None else size,
                                                *a.values()))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 0), (dict(n=0, size=0), 1), (dict(n=0, size=200), 1), (dict(n=-1), 1),
    (dict(d=96), 2), (dict(bs=8), 2), (dict(dtype=3), 2), (dict(hkv=0), 1), (dict(nb=0), 1),
    (dict(n=2 ** 30), 2), (dict(nb=2 ** 27), 2)])
def test_all_refuse(lib, name, kw, status):
    assert _call(lib, name, **kw) == status


def test_no_arguments(lib):
    assert [getattr(lib, x)(None) for x in NAMES] == [1] * 6


@pytest.mark.parametrize("name", [x for x in NAMES if x != "pa_sparse_decode"])
@pytest.mark.parametrize("kw,status", [
    (dict(mb=0), 1), (dict(mb=-3), 1), (dict(mb=2 ** 28), 2), (dict(mb=2 ** 26, n=1, hkv=1), 2),
    (dict(tables=0), 1), (dict(lens=0x1002), 1)])
def test_tables(lib, name, kw, status):
    assert _call(lib, name, **kw) == status


@pytest.mark.parametrize("name,most", [("pa_select_blocks", 16), ("pa_sparse_decode", 16),
                                       ("pa_decode_mass", 16), ("pa_prefill_mass", 128)])
def test_heads(lib, name, most):
    assert _call(lib, name, hq=7) == 1 and _call(lib, name, hq=0) == 1
    assert _call(lib, name, hq=2 * most + 2) == 2
    assert _call(lib, name, hq=2 * most, q=0) == 1                   # served: null refused


@pytest.mark.parametrize("name,kw,status", [
    ("pa_block_bounds", dict(bounds=0), 1), ("pa_block_bounds", dict(k=0x1008), 1),
    ("pa_block_bounds", dict(starts=0x1001), 1),
    ("pa_select_blocks", dict(keep=0), 1), ("pa_select_blocks", dict(last=0), 1),
    ("pa_select_blocks", dict(first=-1), 1), ("pa_select_blocks", dict(first=2, last=3), 1),
    ("pa_select_blocks", dict(first=2 ** 31 - 1, last=2 ** 31 - 1), 1),
    ("pa_select_blocks", dict(bounds=0x1008), 1), ("pa_select_blocks", dict(tiles=0), 1),
    ("pa_select_blocks", dict(tile_lens=0), 1), ("pa_select_blocks", dict(), 3),
    ("pa_select_blocks", dict(ws=0x1000, wb=64), 3),
    ("pa_select_blocks", dict(ws=0x1010, wb=1 << 20), 3),
    ("pa_sparse_decode", dict(keep=0), 1), ("pa_sparse_decode", dict(tiles=0), 1),
    ("pa_sparse_decode", dict(tile_lens=0x1001), 1), ("pa_sparse_decode", dict(v=0), 1),
    ("pa_sparse_decode", dict(out=FAKE), 1), ("pa_sparse_decode", dict(scale=math.nan), 1),
    ("pa_sparse_decode", dict(scale=1e300), 1),
    ("pa_decode_mass", dict(mass=0), 1), ("pa_decode_mass", dict(mass=0x1008), 1),
    ("pa_decode_mass", dict(out=FAKE), 1), ("pa_decode_mass", dict(out=0), 1),
    ("pa_decode_mass", dict(scale=math.inf), 1), ("pa_decode_mass", dict(decay=math.nan), 1),
    ("pa_decode_mass", dict(decay=math.inf), 1),
    ("pa_prefill_mass", dict(scale=0.0), 1), ("pa_prefill_mass", dict(scale=-1.0), 1),
    ("pa_prefill_mass", dict(decay=math.nan), 1), ("pa_prefill_mass", dict(longest=-1), 1),
    ("pa_prefill_mass", dict(longest=0), 0), ("pa_prefill_mass", dict(rows=-1), 1),
    ("pa_prefill_mass", dict(mass=0), 1), ("pa_prefill_mass", dict(q=0x1008), 1),
    ("pa_prefill_mass", dict(start=0), 1), ("pa_prefill_mass", dict(k=0), 1),
    ("pa_evict", dict(first=-1), 1), ("pa_evict", dict(last=-1), 1), ("pa_evict", dict(mass=0), 1),
    ("pa_evict", dict(v=0x1008), 1), ("pa_evict", dict(new_lens=0), 1), ("pa_evict", dict(), 3),
    ("pa_evict", dict(ws=0x1000, wb=4), 3)])
def test_one_refuses(lib, name, kw, status):
    assert _call(lib, name, **kw) == status


def test_workspace_sizes(lib):
    # scores, 4 bytes for 16 of them, and 8 bytes a score in doubt: rows of 16 blocks
    assert lib.pa_select_blocks_workspace_size(4, 2, 8) == 512 + 256 + 1024
    assert lib.pa_select_blocks_workspace_size(0, 2, 8) == 0
    assert lib.pa_evict_workspace_size(4, 2, 8) == 4 * 4 * 2 * 128
    assert lib.pa_evict_workspace_size(4, 0, 8) == 0
    # past 32 bits
    assert lib.pa_evict_workspace_size(64, 8, 65536) == 4 * 64 * 8 * 65536 * 16
    assert lib.pa_decode_mass_workspace_size(4, 7, 2, 128, 8) == 0
    assert lib.pa_sparse_decode_workspace_size(2 ** 20, 2 ** 13, 2 ** 12, 128, 8) == 0
    assert lib.pa_prefill_mass_workspace_size(4, 0, 8, 2, 8) == 0


def test_bindings_refuse_host_tensors():
    import paged_kv_cache_260_gb300 as pa
    q = torch.zeros(2, 8, 64, dtype=torch.float16)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    t, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    tiles, held = torch.zeros(2, 2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)
    mass, b = torch.zeros(2, 2, 32), torch.zeros(4, 2, 2, 64, dtype=torch.float16)
    for call in (lambda: pa.block_bounds(b, k, t, lens),
                 lambda: pa.select_blocks(tiles, held, q, b, t, lens, workspace=mass),
                 lambda: pa.sparse_decode(q, q, k, k, tiles, held, 1.0, workspace=mass),
                 lambda: pa.decode_mass(q, mass, q, k, k, t, lens, 1.0, workspace=mass),
                 lambda: pa.prefill_mass(mass, q, k, t, lens, torch.arange(3).int(), 1, 1.0,
                                         workspace=mass),
                 lambda: pa.evict(k, k, mass, t, lens, lens, workspace=mass)):
        with pytest.raises(ValueError):
            call()


def test_selection_by_hand():
    # one head of two channels, four blocks; bounds [min, max] a channel
    bnd = torch.tensor([[[[-1., 0.], [2., 1.]]], [[[0., 0.], [1., 1.]]], [[[-4., -1.], [0., 0.]]],
                        [[[0., 0.], [0., 0.]]]])
    tables, q = torch.tensor([[2, 0, 1, 3]]), torch.tensor([[[1., -1.]]])
    # the blocks' scores in the order of positions: 2: 0 + 1, 0: 2 + 0, 1: 1 + 0, 3: 0
    for keep, want in ((1, [3]), (2, [0, 3]), (3, [2, 0, 3]), (4, [2, 0, 1, 3])):
        tiles, held = su.select(q, bnd, tables, [50], keep, 0, 1)
        assert tiles[0, 0].tolist() == want and int(held[0, 0]) == 2 + 16 * (keep - 1)
    assert su.select(q, bnd, tables, [50], 3, 1, 1)[0][0, 0].tolist() == [2, 0, 3]
    # equal scores: the lowest position
    assert su.select(q * 0, bnd, tables, [50], 2, 0, 1)[0][0, 0].tolist() == [2, 3]


def test_accounting_by_hand():
    k = torch.zeros(1, 1, 16, 64)
    k[0, 0, 0, 0], k[0, 0, 1, 0] = 1.0, 2.0
    q = torch.zeros(1, 1, 64)
    q[..., 0] = 1.0
    z = math.exp(1) + math.exp(2) + 1
    w = [math.exp(1) / z, math.exp(2) / z, 1 / z]
    mass = torch.full((1, 1, 16), 3.0)
    _, _, got, _ = su.decode_mass(q, mass, k, k, torch.tensor([[0]]), [3], 1.0, 0.5)
    want = [1.5 + w[0], 1.5 + w[1], w[2]] + [3.0] * 13
    assert all(abs(float(a) - b) < 1e-6 for a, b in zip(got[0, 0], want))
    # two rows: the first sees two tokens, the second three
    got, _ = su.prefill_mass(torch.cat([q, q]), mass, k, torch.tensor([[0]]), [3], [0, 2], 1.0, 0.5)
    y = math.exp(1) + math.exp(2)
    want = [1.5 + w[0] + math.exp(1) / y, w[1] + math.exp(2) / y, w[2]] + [3.0] * 13
    assert all(abs(float(a) - b) < 1e-6 for a, b in zip(got[0, 0], want))


def test_eviction_by_hand():
    k = torch.arange(32.).reshape(2, 1, 16, 1).expand(2, 1, 16, 64).clone()
    mass = torch.zeros(1, 1, 32)
    mass[0, 0, :10] = torch.tensor([0., 5., 1., 5., 2., 7., 2., 9., 0., 0.])
    tables = torch.tensor([[1, 0]])
    # ten tokens to six: the last two stay, and 7, 5 and the first 5s: slots 7, 5, 1, 3
    kk, _, m = su.evict(k, k, mass, tables, [10], [6], 0, 2)
    # slots 5 and 7 lie past the last ones' new place (4, 5) and move to the holes 0 and 2
    assert (kk[1, 0, :10, 0] - 16).tolist() == [5, 1, 7, 3, 8, 9, 6, 7, 8, 9]
    assert m[0, 0, :6].tolist() == [7., 5., 9., 5., 0., 0.]
    kk, _, _ = su.evict(k, k, mass, tables, [10], [6], 1, 2)
    assert (kk[1, 0, :6, 0] - 16).tolist() == [0, 1, 5, 7, 8, 9]
    kk, _, _ = su.evict(k, k, mass, tables, [10], [0], 1, 2)
    assert torch.equal(kk, k)
