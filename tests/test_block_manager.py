"""Host block manager (free list, reference counts, on-demand allocation,
copy-on-write).  CPU only: the manager is host code in the library."""
import json
import os

import numpy as np
import pytest

from paged_kv_cache_260_gb300 import PagedAttnError
from paged_kv_cache_260_gb300.block_manager import PA_ERR_OUT_OF_BLOCKS, BlockManager

GOLDEN = os.path.join(os.path.dirname(__file__), "golden")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_cache_260_gb300 import _build
    _build.build()


def test_page3_pool_state_from_on_demand_allocation():
    # The block-pool figure shows A in blocks 0,2,6, B in 1,4,7 and blocks 3, 5
    # empty.  Reading: a third request C took blocks while A and B grew and has
    # finished; allocating on demand in this order and releasing C gives exactly
    # the printed pool row.
    g = json.load(open(os.path.join(GOLDEN, "page3_block_table.json")))
    bm = BlockManager(g["pool_blocks"], g["block_size"])
    ids = {"A": 1, "B": 2, "C": 3}
    for r in ids.values():
        bm.add_sequence(r)
    for req in ["A", "B", "A", "C", "B", "C", "A", "B"]:     # one block's worth of tokens each
        bm.append(ids[req], g["block_size"])
    bm.free(ids["C"])
    for req in ("A", "B"):
        table, nb, ln = bm.block_table(ids[req], 3)
        assert table.tolist() == g["tables"][req] and nb == 3 and ln == 48
    st = bm.stats()
    assert st["free_blocks"] == len(g["free_blocks"])
    assert [b for b in range(g["pool_blocks"]) if bm.ref_count(b) == 0] == g["free_blocks"]


def test_waste_under_one_block_and_slots_follow_the_table():
    rng = np.random.default_rng(0)
    bm = BlockManager(4000)
    lens = {}
    for sid in range(60):
        bm.add_sequence(sid)
        lens[sid] = 0
    for _ in range(400):
        sid = int(rng.integers(60))
        n = int(rng.integers(1, 40))
        slots, cow = bm.append(sid, n)
        assert cow is None
        table, nb, ln = bm.block_table(sid, 256)
        for i, sl in enumerate(slots):
            t = lens[sid] + i
            assert sl == table[t // 16] * 16 + t % 16
        lens[sid] += n
        assert ln == lens[sid] and nb == -(-ln // 16)       # under one block of waste
    st = bm.stats()
    assert st["num_blocks"] - st["free_blocks"] == sum(-(-L // 16) for L in lens.values())


def test_out_of_blocks_changes_nothing():
    bm = BlockManager(4)
    bm.add_sequence(0)
    bm.append(0, 40)                                        # 3 blocks
    before = bm.stats()
    with pytest.raises(PagedAttnError) as e:
        bm.append(0, 40)                                    # needs 3 more, 1 free
    assert e.value.status == PA_ERR_OUT_OF_BLOCKS
    assert bm.stats() == before and bm.block_table(0, 8)[2] == 40
    bm.append(0, 8)                                         # fits the partial block + 1 new


def test_fork_and_copy_on_write():
    bm = BlockManager(64)
    bm.add_sequence(0)
    bm.append(0, 40)                                        # blocks 0,1,2; block 2 half full
    for c in (1, 2, 3):
        bm.fork(0, c)
    assert [bm.ref_count(b) for b in (0, 1, 2)] == [4, 4, 4]
    slots, cow = bm.append(1, 1)                            # write into the shared block
    assert cow == (2, 3)                                    # copy of block 2 into fresh block 3
    assert slots[0] == 3 * 16 + 8
    assert bm.ref_count(2) == 3 and bm.ref_count(3) == 1
    assert bm.append(1, 1)[1] is None                       # its own copy now
    assert bm.append(2, 1)[1] == (2, 4)
    assert bm.append(0, 1)[1] == (2, 5)                     # the parent copies too
    slots, cow = bm.append(3, 1)                            # last sharer keeps the original
    assert cow is None and slots[0] == 2 * 16 + 8
    assert bm.stats()["cow_copies"] == 3
    for sid in range(4):                                    # prompt blocks still shared
        assert bm.block_table(sid, 4)[0][:2].tolist() == [0, 1]


def test_block_aligned_prompt_needs_no_copy():
    bm = BlockManager(64)
    bm.add_sequence(0)
    bm.append(0, 32)
    bm.fork(0, 1)
    slots, cow = bm.append(1, 1)
    assert cow is None and slots[0] // 16 not in (0, 1)
    assert bm.ref_count(0) == 2 and bm.ref_count(1) == 2


def test_no_leak_and_reference_invariant():
    rng = np.random.default_rng(1)
    bm = BlockManager(3000)
    live = []
    for step in range(600):
        op = rng.integers(4)
        if op == 0 or not live:
            sid = step
            bm.add_sequence(sid)
            live.append(sid)
        elif op == 1:
            child = 100000 + step
            bm.fork(int(rng.choice(live)), child)
            live.append(child)
        elif op == 2:
            sid = int(rng.choice(live))
            slots, cow = bm.append(sid, int(rng.integers(1, 20)))
            # the block written to is owned by this sequence alone
            assert bm.ref_count(int(slots[-1]) // 16) == 1
        else:
            sid = live.pop(int(rng.integers(len(live))))
            bm.free(sid)
        total_refs = sum(bm.ref_count(b) for b in range(3000))
        assert total_refs == sum(bm.block_table(s, 256)[1] for s in live)
    for sid in live:
        bm.free(sid)
    st = bm.stats()
    assert st["free_blocks"] == 3000 and st["allocations"] == st["releases"]
    assert st["shared_blocks"] == 0 and st["num_sequences"] == 0


def test_a_shortened_sequence_goes_on_from_its_new_length():
    bm = BlockManager(16)
    bm.add_sequence(0)
    bm.append(0, 70)                                        # blocks 0 to 4
    bm.shorten(0, 40)
    table, nb, ln = bm.block_table(0, 6)
    assert table.tolist() == [0, 1, 2, -1, -1, -1] and nb == 3 and ln == 40
    st = bm.stats()
    assert st["free_blocks"] == 13 and st["releases"] == 2
    slots, cow = bm.append(0, 10)                           # 8 more of block 2, then block 3 again
    assert cow is None and slots.tolist() == [2 * 16 + 8 + i for i in range(8)] + [48, 49]
    bm.shorten(0, 50)                                       # its own length, and more: as it was
    bm.shorten(0, 2 ** 62)
    assert bm.block_table(0, 6)[1:] == (4, 50)
    bm.shorten(0, 48)                                       # on a block's border
    assert bm.block_table(0, 6)[1:] == (3, 48) and bm.append(0, 1)[0][0] == 48
    bm.shorten(0, 0)
    assert bm.block_table(0, 6)[1:] == (0, 0) and bm.stats()["free_blocks"] == 16
    assert bm.append(0, 1)[0][0] == 0


def test_shortening_keeps_what_others_hold():
    bm = BlockManager(16)
    bm.add_sequence(0)
    bm.append(0, 70)
    bm.fork(0, 1)
    bm.shorten(1, 20)
    assert [bm.ref_count(b) for b in range(5)] == [2, 2, 1, 1, 1]
    assert bm.stats()["free_blocks"] == 11 and bm.block_table(0, 5)[1:] == (5, 70)
    slots, cow = bm.append(1, 1)                            # into the shared, partly held block
    assert cow == (1, 5) and slots[0] == 5 * 16 + 4
    bm.free(0)
    bm.free(1)
    assert bm.stats()["free_blocks"] == 16


def test_own_blocks_copies_the_shared_ones_of_the_first_tokens():
    bm = BlockManager(16)
    bm.add_sequence(0)
    bm.append(0, 70)                                        # blocks 0 to 4
    assert bm.own_blocks(0, 70).shape == (0, 2)             # nothing is shared
    bm.fork(0, 1)
    assert bm.append(1, 1)[1] == (4, 5)                     # block 4 is not any more
    pairs = bm.own_blocks(1, 33)                            # three blocks hold them
    assert pairs.tolist() == [[0, 6], [1, 7], [2, 8]]
    assert bm.block_table(1, 5)[0].tolist() == [6, 7, 8, 3, 5]
    assert bm.block_table(0, 5)[0].tolist() == [0, 1, 2, 3, 4]
    assert [bm.ref_count(b) for b in range(9)] == [1, 1, 1, 2, 1, 1, 1, 1, 1]
    assert bm.stats()["cow_copies"] == 4
    assert len(bm.own_blocks(1, 48)) == 0 and len(bm.own_blocks(1, 0)) == 0
    assert bm.own_blocks(0, 1000).tolist() == [[3, 9]]      # more than it has: all of them
    assert all(bm.ref_count(b) == 1 for b in range(10))


def test_own_blocks_refused_changes_nothing():
    import ctypes as C
    bm = BlockManager(6)
    bm.add_sequence(0)
    bm.append(0, 64)
    bm.fork(0, 1)
    before = bm.stats()
    with pytest.raises(PagedAttnError) as e:
        bm.own_blocks(1, 64)                                # four copies, two free blocks
    assert e.value.status == PA_ERR_OUT_OF_BLOCKS and bm.stats() == before
    n, pairs = C.c_int(-1), np.zeros(4, np.int64)
    assert bm._L.pa_bm_own_blocks(bm._h, 1, 40, pairs.ctypes.data, 2, C.byref(n)) == 1
    assert n.value == 3 and bm.stats() == before            # room for two
    assert bm._L.pa_bm_own_blocks(bm._h, 1, 40, None, 0, C.byref(n)) == 1 and n.value == 3
    assert bm._L.pa_bm_own_blocks(bm._h, 1, 40, None, 2, C.byref(n)) == 1
    assert bm._L.pa_bm_own_blocks(bm._h, 1, 40, pairs.ctypes.data, 2, None) == 1
    for call in (lambda: bm.own_blocks(7, 3), lambda: bm.own_blocks(1, -1),
                 lambda: bm.shorten(7, 3), lambda: bm.shorten(1, -1)):
        with pytest.raises(PagedAttnError):
            call()
    assert bm.stats() == before and len(bm.own_blocks(1, 32)) == 2


def test_no_leak_with_shortened_and_owned_sequences():
    rng = np.random.default_rng(3)
    bm = BlockManager(3000)
    live = {}
    for step in range(800):
        op = int(rng.integers(6))
        if op == 0 or not live:
            bm.add_sequence(step)
            live[step] = 0
        elif op == 1:
            parent = int(rng.choice(list(live)))
            bm.fork(parent, 100000 + step)
            live[100000 + step] = live[parent]
        elif op == 2:
            sid, n = int(rng.choice(list(live))), int(rng.integers(1, 60))
            slots, _ = bm.append(sid, n)
            table = bm.block_table(sid, 3000)[0]
            assert slots.tolist() == [table[t // 16] * 16 + t % 16
                                      for t in range(live[sid], live[sid] + n)]
            live[sid] += n
        elif op == 3:
            sid = int(rng.choice(list(live)))
            n = int(rng.integers(0, live[sid] + 5))
            bm.shorten(sid, n)
            live[sid] = min(live[sid], n)
        elif op == 4:
            sid = int(rng.choice(list(live)))
            n = int(rng.integers(0, live[sid] + 5))
            pairs = bm.own_blocks(sid, n)
            table = bm.block_table(sid, 3000)[0]
            own = -(-min(n, live[sid]) // 16)
            assert all(bm.ref_count(int(b)) == 1 for b in table[:own])
            assert set(pairs[:, 1].tolist()) <= set(table[:own].tolist())
        else:
            sid = int(rng.choice(list(live)))
            bm.free(sid)
            del live[sid]
        assert [bm.block_table(s, 3000)[1:] for s in live] == [(-(-n // 16), n)
                                                               for n in live.values()]
        assert (sum(bm.ref_count(b) for b in range(3000)) == sum(-(-n // 16)
                                                                 for n in live.values()))
    for sid in live:
        bm.free(sid)
    st = bm.stats()
    assert st["free_blocks"] == 3000 and st["allocations"] == st["releases"]


def test_bad_calls():
    bm = BlockManager(8)
    bm.add_sequence(5)
    with pytest.raises(PagedAttnError):
        bm.add_sequence(5)
    with pytest.raises(PagedAttnError):
        bm.append(6, 1)
    with pytest.raises(PagedAttnError):
        bm.fork(7, 8)
    with pytest.raises(PagedAttnError):
        bm.block_table(5, 0) if bm.append(5, 20) else None    # 2 blocks do not fit 0 entries
    assert bm.ref_count(99) == -1
    with pytest.raises(ValueError):
        BlockManager(0)
