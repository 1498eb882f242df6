"""Decode steps driven by the host block manager: prompts are written, forked
into samples, and every step appends one token per sample.  The manager's
copy-on-write pairs go to copy_blocks and its slots to decode_append.  Each
step is checked against the oracle run on a host replica of the pool; at the
end the pools are bit-identical and freeing every sequence leaks nothing."""
import numpy as np
import pytest
import torch

import oracle
import sparse_util as su
import synth
from gpu_util import TOL, dev_bits, host_bits, max_err
from paged_kv_cache_260_gb300.block_manager import BlockManager

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt_lens,mode", [((40, 37), 0), ((32, 50), -1), ((40, 37), 16)])
def test_parallel_sampling_steps_with_the_block_manager(pa, prompt_lens, mode):
    rng = np.random.default_rng(7)
    NB, HKV, HQ, D, S, STEPS, MAXB = 96, 2, 8, 128, 4, 6, 8
    dt = "f16"

    def bits(*shape):
        return synth.to_bits(rng.standard_normal(shape).astype(np.float32), dt)

    k_host = bits(NB, HKV, 16, D)                            # stale contents everywhere
    v_host = bits(NB, HKV, 16, D)
    k_dev, v_dev = dev_bits(k_host, dt), dev_bits(v_host, dt)
    bm = BlockManager(NB)
    samples = []
    for p, L in enumerate(prompt_lens):
        root = 1000 * p
        bm.add_sequence(root)
        slots, cow = bm.append(root, L)
        assert cow is None
        kn, vn = bits(L, HKV, D), bits(L, HKV, D)
        pa.reshape_and_cache(dev_bits(kn, dt), dev_bits(vn, dt), k_dev, v_dev,
                             torch.from_numpy(slots).cuda())
        oracle.reshape_and_cache(k_host, v_host, kn, vn, slots)
        samples.append(root)
        for c in range(1, S):
            bm.fork(root, root + c)
            samples.append(root + c)
    n = len(samples)
    for step in range(STEPS):
        slots = np.empty(n, np.int64)
        pairs = []
        for i, sid in enumerate(samples):
            sl, cow = bm.append(sid, 1)
            slots[i] = sl[0]
            if cow is not None:
                pairs.append(cow)
        tables = np.stack([bm.block_table(sid, MAXB)[0] for sid in samples])
        lens = np.array([bm.block_table(sid, MAXB)[2] for sid in samples], np.int32)
        q, kn, vn = bits(n, HQ, D), bits(n, HKV, D), bits(n, HKV, D)
        if pairs:
            bmap = np.array(pairs, np.int64)
            pa.copy_blocks(k_dev, v_dev, torch.from_numpy(bmap).cuda())
            oracle.copy_blocks(k_host, v_host, bmap)
        out = torch.empty(n, HQ, D, dtype=torch.float16, device="cuda")
        pa.decode_append(out, dev_bits(q, dt), k_dev, v_dev, torch.from_numpy(tables).cuda(),
                         torch.from_numpy(lens).cuda(), dev_bits(kn, dt), dev_bits(vn, dt),
                         torch.from_numpy(slots).cuda(), 1 / np.sqrt(D), partition_size=mode)
        oracle.reshape_and_cache(k_host, v_host, kn, vn, slots)
        ref = oracle.decode(q, k_host, v_host, tables, lens, 1 / np.sqrt(D), dt)
        assert max_err(out, ref) <= TOL[dt], f"step {step}"
        assert pa.get_device_error() == 0
        if step == 0:
            # first token after an unaligned prompt: every sample but the last to
            # write copies the shared partial block
            unaligned = sum(1 for L in prompt_lens if L % 16)
            assert len(pairs) == unaligned * (S - 1)
    assert np.array_equal(host_bits(k_dev), k_host) and np.array_equal(host_bits(v_dev), v_host)
    for sid in samples:
        bm.free(sid)
    st = bm.stats()
    assert st["free_blocks"] == NB and st["allocations"] == st["releases"]


def test_evicted_sequences_go_on_with_the_block_manager(pa):
    """Forked prompts are cut to their heaviest tokens and decoded on: the manager copies the
    shared blocks first, takes back the blocks past the new ends and hands out slots from there."""
    r = torch.Generator().manual_seed(11)
    hq, hkv, d, nb, mb, scale, budget = 8, 2, 64, 64, 24, 0.125, 100

    def rows(*shape):
        return torch.randn(*shape, generator=r).half()

    k, v = rows(nb, hkv, 16, d).cuda(), rows(nb, hkv, 16, d).cuda()
    bm = BlockManager(nb)
    for sid, length in ((0, 300), (2, 220)):
        bm.add_sequence(sid)
        slots, _ = bm.append(sid, length)
        pa.reshape_and_cache(rows(length, hkv, d).cuda(), rows(length, hkv, d).cuda(), k, v,
                             torch.from_numpy(slots).cuda())
    bm.fork(0, 1)                                            # 0 stays whole
    bm.fork(2, 3)
    ids = [1, 2, 3]

    def state():
        t = np.stack([bm.block_table(s, mb)[0] for s in ids])
        return torch.from_numpy(t), [bm.block_table(s, mb)[2] for s in ids]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    whole = [su.rows_of(x.cpu(), torch.from_numpy(bm.block_table(0, mb)[0]), 300, h)
             for x in (k, v) for h in range(hkv)]
    tables, lens = state()
    mass = torch.full((3, hkv, 16 * mb), np.nan).cuda()
    q = rows(24, hq, d)
    pa.prefill_mass(mass, q.cuda(), k, tables.cuda(), ints(lens), ints([0, 8, 16, 24]), 8, scale,
                    decay=0.0)
    for _ in range(2):
        pairs = np.concatenate([bm.own_blocks(s, budget) for s in ids])
        if len(pairs):
            pa.copy_blocks(k, v, torch.from_numpy(pairs).cuda())
        assert len(pairs) in (0, 14)                         # 7 blocks of 1 and of 2 or 3
        tables, lens = state()
        before = k.cpu(), v.cpu(), mass.cpu()
        pa.evict(k, v, mass, tables.cuda(), ints(lens), ints([budget] * 3), keep_first=4,
                 keep_last=16)
        ref = su.evict(*before, tables, lens, [budget] * 3, 4, 16)
        assert all(torch.equal(su.bits(x), su.bits(y)) for x, y in zip((k, v, mass), ref))
        for s in ids:
            bm.shorten(s, budget)
        assert state()[1] == [budget] * 3
        for step in range(20):
            new = [bm.append(s, 1) for s in ids]
            assert all(cow is None for _, cow in new)
            slots = torch.from_numpy(np.concatenate([x for x, _ in new]))
            pa.reshape_and_cache(rows(3, hkv, d).cuda(), rows(3, hkv, d).cuda(), k, v, slots.cuda())
            tables, lens = state()
            q, before = rows(3, hq, d), mass.cpu()
            out, _ = pa.decode_mass(torch.empty_like(q).cuda(), mass, q.cuda(), k, v, tables.cuda(),
                                    ints(lens), scale)
            ref = su.decode_mass(q, before, k.cpu(), v.cpu(), tables, lens, scale, 1.0)
            su.close(out, *ref[:2], "step")
            su.mass_close(mass, *ref[2:], "step")
        assert lens == [budget + 20] * 3
    assert pa.get_device_error() == 0
    # the sequence that was not cut has its tokens still
    now = [su.rows_of(x.cpu(), torch.from_numpy(bm.block_table(0, mb)[0]), 300, h)
           for x in (k, v) for h in range(hkv)]
    assert all(torch.equal(x, y) for x, y in zip(whole, now))
    for s in [0] + ids:
        bm.free(s)
    assert bm.stats()["free_blocks"] == nb
