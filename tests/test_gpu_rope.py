"""rope_and_cache and qk_norm_rope against the formula in 64 bits.

Tolerance, element by element, derived before the first run.  The kernel
computes in fp32 and rounds once: a rounding is off by at most eps/2 of the
value.  Before it, a rotated channel a cos - b sin carries the relative errors
of its terms: the norm's factor (a sum of at most 128 squares in a tree no
deeper than 16 + 3 steps, halved by the root; an approximate reciprocal root
good to 2^-22; two products) and the rotation's three roundings, together
below 30 * 2^-24 < 2^-19 of |a| + |b|, which 2^-18 covers with the second-order
terms; half the smallest fp16 subnormal, 2^-25, covers results below the normal
range.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import TORCH_DTYPE, TOL

pytestmark = pytest.mark.gpu

EPS = 1e-5


def table(n, rot, theta=10000.0):
    a = torch.arange(n).double()[:, None] * theta ** (-torch.arange(0, rot, 2).double() / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def reference(x, w, cos_sin, pos, maps, inter):
    """The formula in 64 bits, and each channel's |a| + |b|."""
    x = x.double().cpu()
    t, h, d = x.shape
    seg, rot = d // maps, cos_sin.shape[1]
    y = x.reshape(t, h, maps, seg)
    if w is not None:
        y = y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + EPS) * w.double().cpu()
    cs = cos_sin.double().cpu()[pos.long().cpu().clamp(0, cos_sin.shape[0] - 1)]
    out, mag = y.clone(), y.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = cs[:, i, None, None], cs[:, rot // 2 + i, None, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    return out.reshape(t, h, d), mag.reshape(t, h, d)


def close(got, ref, mag, what):
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + 2.0 ** -18 * mag + 2.0 ** -25
    d = (got.double().cpu() - ref).abs()
    assert bool((d <= tol).all()), f"{what}: off by {float((d / tol).max())} of the tolerance"


class Tokens:
    def __init__(self, t, hq, hkv, d, dtype, maps=1, rot=None, norm="qk", fused=False, npos=300,
                 seed=0, pool=True):
        g = torch.Generator().manual_seed(seed)
        dt = TORCH_DTYPE[dtype]
        rnd = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
        if fused:
            x = rnd(t, (hq + 2 * hkv) * d + 24)              # a wider row than the three need
            self.q = x[:, :hq * d].view(t, hq, d)
            self.k = x[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
            self.v = x[:, (hq + hkv) * d:(hq + 2 * hkv) * d].view(t, hkv, d)
        else:
            self.q, self.k, self.v = rnd(t, hq, d), rnd(t, hkv, d), rnd(t, hkv, d)
        rot = d // maps if rot is None else rot
        self.cs = table(npos, rot).cuda()
        self.pos = torch.randint(0, npos, (t,), generator=g).int().cuda()
        w = lambda: (1 + 0.3 * torch.randn(d // maps, generator=g)).to(dt).cuda()  # noqa: E731
        self.qw, self.kw = (w() if c in norm else None for c in "qk")
        self.q_out = torch.full((t, hq, d), 7.0, dtype=dt, device="cuda")
        self.maps = maps
        if pool:
            self.nb = t + 3
            self.kc, self.vc = (rnd(self.nb, hkv, 16, d) for _ in range(2))
            self.slots = torch.randperm(self.nb * 16, generator=g)[:t].cuda()

    def append(self, pa, inter=False, **kw):
        pa.rope_and_cache(self.q_out, self.q, self.k, self.v, self.kc, self.vc, self.slots,
                          self.pos, self.cs, q_norm=self.qw, k_norm=self.kw, eps=EPS,
                          interleaved=inter, num_maps=self.maps, **kw)

    def check(self, pa, run, inter=False, skipped=()):
        """Runs the append and checks q_out and every byte of both pools."""
        kc, vc, q_in, k_in = self.kc.clone(), self.vc.clone(), self.q.clone(), self.k.clone()
        before = self.q_out.clone()
        run()
        torch.cuda.synchronize()
        live = torch.ones(len(self.pos), dtype=torch.bool)
        live[list(skipped)] = False
        rq, mq = reference(q_in, self.qw, self.cs, self.pos, self.maps, inter)
        rk, mk = reference(k_in, self.kw, self.cs, self.pos, self.maps, inter)
        close(self.q_out.cpu()[live], rq[live], mq[live], "q")
        assert torch.equal(self.q_out.cpu()[~live], before.cpu()[~live])
        s = self.slots.cpu()[live]
        got_k = self.kc[(s // 16).cuda(), :, (s % 16).cuda()].cpu()
        close(got_k, rk[live], mk[live], "k")
        kc[(s // 16).cuda(), :, (s % 16).cuda()] = got_k.cuda()
        vc[(s // 16).cuda(), :, (s % 16).cuda()] = self.v[live.cuda()]
        bits = lambda x: x.contiguous().view(torch.int16)  # noqa: E731
        assert torch.equal(bits(self.kc), bits(kc)), "other key slots changed"
        assert torch.equal(bits(self.vc), bits(vc)), "values"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,dtype,maps,rot,norm,fused", [
    (1, 8, 8, 64, "f16", 1, 64, "", False), (1, 1, 1, 128, "bf16", 1, 16, "qk", True),
    (2, 3, 1, 64, "bf16", 1, 48, "qk", True), (5, 32, 8, 128, "bf16", 1, 128, "qk", True),
    (37, 10, 2, 128, "f16", 1, 96, "q", False), (64, 32, 32, 128, "f16", 1, 128, "k", False),
    (3, 8, 2, 64, "f16", 2, 32, "qk", False), (19, 5, 5, 64, "bf16", 2, 16, "qk", True),
    (130, 20, 4, 128, "bf16", 2, 64, "qk", False), (41, 7, 7, 128, "f16", 2, 48, "", True),
    (1500, 40, 8, 128, "f16", 1, 64, "qk", True), (2777, 9, 3, 64, "bf16", 1, 32, "qk", True)])
def test_append(pa, t, hq, hkv, d, dtype, maps, rot, norm, fused, inter):
    x = Tokens(t, hq, hkv, d, dtype, maps, rot, norm, fused, seed=t)
    x.check(pa, lambda: x.append(pa, inter), inter)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,dtype,maps,rot,norm,fused", [
    (1, 8, 2, 128, "bf16", 1, 128, "qk", False), (77, 12, 4, 64, "f16", 1, 32, "qk", True),
    (300, 16, 2, 128, "f16", 2, 64, "", True), (33, 5, 1, 64, "bf16", 2, 32, "qk", False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_qk_norm_rope(pa, t, hq, hkv, d, dtype, maps, rot, norm, fused, inter, in_place):
    x = Tokens(t, hq, hkv, d, dtype, maps, rot, norm, fused, seed=t + 1, pool=False)
    if t > 3:
        x.pos[2] = -1
    rq, mq = reference(x.q, x.qw, x.cs, x.pos, maps, inter)
    rk, mk = reference(x.k, x.kw, x.cs, x.pos, maps, inter)
    v = x.v.clone()
    qo = x.q if in_place else x.q_out
    ko = x.k if in_place else torch.full_like(x.k, 7.0)
    q2, k2 = qo.clone(), ko.clone()
    pa.qk_norm_rope(qo, ko, x.q, x.k, x.pos, x.cs, q_norm=x.qw, k_norm=x.kw, eps=EPS,
                    interleaved=inter, num_maps=maps)
    live = (x.pos >= 0).cpu()
    close(qo.cpu()[live], rq[live], mq[live], "q")
    close(ko.cpu()[live], rk[live], mk[live], "k")
    assert torch.equal(qo.cpu()[~live], q2.cpu()[~live])
    assert torch.equal(ko.cpu()[~live], k2.cpu()[~live])
    assert torch.equal(x.v, v)                               # the rest of a fused row
    assert pa.get_device_error() == 0


# Enough tokens for the kernel that copies rows through shared memory: with a
# few units of work a warp, and with so many that the last are handed out apart.
@pytest.mark.parametrize("t,hq,hkv,d,dtype,maps,rot,norm,fused,inter", [
    (5003, 32, 8, 128, "bf16", 1, 128, "qk", True, False),
    (7001, 10, 2, 128, "f16", 1, 96, "k", False, True),
    (11003, 6, 3, 64, "bf16", 2, 16, "qk", True, False),
    (13001, 9, 3, 64, "f16", 1, 64, "", False, True),
    (80111, 1, 1, 64, "f16", 1, 48, "q", True, False),
    (81001, 1, 1, 128, "bf16", 2, 64, "qk", False, True)])
def test_append_many(pa, t, hq, hkv, d, dtype, maps, rot, norm, fused, inter):
    x = Tokens(t, hq, hkv, d, dtype, maps, rot, norm, fused, seed=t)
    skipped = [0, 1, 17, t // 2, t - 1]
    x.slots[0], x.slots[17], x.pos[t // 2] = -1, -7, -1
    x.pos[1], x.slots[t - 1] = 300, x.nb * 16               # outside the table, the pool
    x.check(pa, lambda: x.append(pa, inter), inter, skipped=skipped)
    assert pa.get_device_error() == pa.DEVERR["POSITION_RANGE"] | pa.DEVERR["SLOT_RANGE"]


@pytest.mark.parametrize("t,hq,hkv,d,dtype,inter", [(9001, 12, 4, 64, "f16", False),
                                                    (4001, 32, 8, 128, "bf16", True)])
def test_qk_norm_rope_many_in_place(pa, t, hq, hkv, d, dtype, inter):
    x = Tokens(t, hq, hkv, d, dtype, seed=t, fused=True, pool=False)
    rq, mq = reference(x.q, x.qw, x.cs, x.pos, 1, inter)
    rk, mk = reference(x.k, x.kw, x.cs, x.pos, 1, inter)
    v = x.v.clone()
    pa.qk_norm_rope(x.q, x.k, x.q, x.k, x.pos, x.cs, q_norm=x.qw, k_norm=x.kw, eps=EPS,
                    interleaved=inter)
    close(x.q, rq, mq, "q")
    close(x.k, rk, mk, "k")
    assert torch.equal(x.v, v) and pa.get_device_error() == 0


def test_padding_and_bad_entries_are_skipped(pa):
    x = Tokens(40, 8, 2, 128, "bf16", seed=3, fused=True)
    x.slots[4] = -1
    x.slots[17] = -(1 << 40)
    x.pos[20] = -5
    x.check(pa, lambda: x.append(pa), skipped=[4, 17, 20])
    assert pa.get_device_error() == 0
    for tensor, at, value, bit in ((x.pos, 9, 300, "POSITION_RANGE"),
                                   (x.pos, 9, 2 ** 31 - 1, "POSITION_RANGE"),
                                   (x.slots, 11, x.nb * 16, "SLOT_RANGE"),
                                   (x.slots, 11, 1 << 40, "SLOT_RANGE")):
        keep = tensor[at].clone()
        tensor[at] = value
        x.check(pa, lambda: x.append(pa), skipped=[4, 17, 20, at])
        assert pa.get_device_error() == pa.DEVERR[bit]
        tensor[at] = keep
    # a padding token's bad position is not looked at
    x.pos[4] = 10 ** 6
    x.check(pa, lambda: x.append(pa), skipped=[4, 17, 20])
    assert pa.get_device_error() == 0


def test_values_are_raw_bits_and_bad_rows_stay_apart(pa):
    x = Tokens(6, 4, 2, 64, "f16", seed=5, norm="qk")
    x.v.view(torch.int16)[2] = torch.arange(0x7c01, 0x7c01 + 64).short().cuda()   # NaN payloads
    x.q[1, 0, 3] = float("inf")                              # one head of one token
    x.k[5] = 0                                               # a row of zeros: 0 / sqrt(eps)
    q_ok = torch.ones(6, 4, dtype=torch.bool)
    q_ok[1, 0] = False
    clean = Tokens(6, 4, 2, 64, "f16", seed=5, norm="qk")
    clean.k[5] = 0
    clean.append(pa)
    x.append(pa)
    torch.cuda.synchronize()
    assert torch.equal(x.q_out.cpu()[q_ok], clean.q_out.cpu()[q_ok])
    assert torch.equal(x.kc, clean.kc)
    s = x.slots[5]
    assert bool((x.kc[s // 16, :, s % 16] == 0).all())
    s = x.slots[2]
    assert torch.equal(x.vc.view(torch.int16)[s // 16, :, s % 16], x.v.view(torch.int16)[2])


def test_far_positions(pa):
    # angles of far positions are as exact as the table's
    x = Tokens(8, 4, 2, 128, "f16", seed=6, npos=200000)
    x.pos.copy_(torch.tensor([0, 1, 131071, 199999, 65537, 99999, 4096, 2]).int())
    x.check(pa, lambda: x.append(pa))


def test_bit_stable_over_batches(pa):
    # a token's result does not depend on the tokens beside it, or on their number
    big = Tokens(12000, 12, 4, 128, "bf16", seed=7)
    big.append(pa)
    for n in (1, 3, 64, 700):
        out = torch.full_like(big.q_out[:n], 7.0)
        kc, vc = big.kc.clone(), big.vc.clone()
        pa.rope_and_cache(out, big.q[:n], big.k[:n], big.v[:n], kc, vc, big.slots[:n],
                          big.pos[:n], big.cs, q_norm=big.qw, k_norm=big.kw, eps=EPS)
        assert torch.equal(out, big.q_out[:n]) and torch.equal(kc, big.kc)


def test_graph_replay_and_other_stream(pa):
    x = Tokens(50, 8, 2, 128, "bf16", seed=8, fused=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x.append(pa)                                         # warm up
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.append(pa)
    # new inputs in the captured buffers, as a serving loop feeds them
    y = Tokens(50, 8, 2, 128, "bf16", seed=9, fused=True)
    for a, b in ((x.q, y.q), (x.k, y.k), (x.v, y.v), (x.pos, y.pos), (x.slots, y.slots)):
        a.copy_(b)
    x.check(pa, g.replay)
    # an explicit stream
    y.append(pa, stream=s)
    s.synchronize()
    z = Tokens(50, 8, 2, 128, "bf16", seed=9, fused=True)
    z.append(pa)
    assert torch.equal(z.q_out, y.q_out) and torch.equal(z.kc, y.kc)


def test_binding_refusals(pa):
    x = Tokens(4, 8, 2, 64, "f16")
    args = lambda **kw: {**dict(q_out=x.q_out, q=x.q, k_new=x.k, v_new=x.v,  # noqa: E731
                                k_cache=x.kc,
                                v_cache=x.vc, slot_mapping=x.slots, positions=x.pos,
                                cos_sin=x.cs), **kw}
    bad = [dict(q=x.q.cpu()), dict(positions=x.pos.long()), dict(slot_mapping=x.slots.int()),
           dict(cos_sin=x.cs.half()), dict(cos_sin=x.cs.cpu()), dict(k_new=x.k[:3]),
           dict(v_new=x.v.bfloat16()), dict(k_cache=x.kc.bfloat16()), dict(q_out=x.q_out[:, :4]),
           dict(q=x.q.transpose(0, 1).contiguous().transpose(0, 1)),  # heads apart
           dict(q_norm=torch.ones(32, dtype=torch.float16, device="cuda")),
           dict(q_norm=torch.ones(64, device="cuda")), dict(v_cache=x.vc[:, :1]),
           dict(q=x.q[:, :, ::2].repeat(1, 1, 2)[:, :, ::1].float())]
    before = x.kc.clone()
    for kw in bad:
        with pytest.raises(ValueError):
            pa.rope_and_cache(**args(**kw))
    for kw in (dict(num_maps=3), dict(num_maps=2), dict(eps=-1.0)):
        with pytest.raises(pa.PagedAttnError):
            pa.rope_and_cache(**args(**kw))
    torch.cuda.synchronize()
    assert torch.equal(before, x.kc) and bool((x.q_out == 7).all())
    pa.rope_and_cache(x.q_out[:0], x.q[:0], x.k[:0], x.v[:0], x.kc, x.vc, x.slots[:0], x.pos[:0],
                      x.cs)                                  # no tokens: nothing to do


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_then_decode(pa, dtype):
    """A prompt written by rope_and_cache and attended by prefill, then decode steps whose
    tokens go through rope_and_cache and through qk_norm_rope + decode_append, each
    attention checked against the oracle on the pool's own contents."""
    hq, hkv, d, n = 8, 2, 128, 3
    lens = [37, 1, 100]
    maxb = 9
    scale = d ** -0.5
    g = torch.Generator().manual_seed(11)
    tables = torch.randperm(n * maxb + 4, generator=g)[:n * maxb].view(n, maxb).int().cuda()
    total = sum(lens)
    x = Tokens(total, hq, hkv, d, dtype, seed=12, fused=True)
    x.nb = n * maxb + 4
    x.kc = torch.zeros(x.nb, hkv, 16, d, dtype=x.q.dtype, device="cuda")
    x.vc = torch.zeros_like(x.kc)
    where = [(s, i) for s, L in enumerate(lens) for i in range(L)]
    x.pos = torch.tensor([i for _, i in where]).int().cuda()
    x.slots = torch.stack([tables[s, i // 16].long() * 16 + i % 16 for s, i in where])
    x.check(pa, lambda: x.append(pa))
    start = torch.tensor(np.cumsum([0] + lens)).int().cuda()
    out = torch.empty_like(x.q_out)
    pa.prefill(out, x.q_out, x.kc, x.vc, tables, torch.tensor(lens).int().cuda(), start, max(lens),
               scale)

    def host(t):
        return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)

    ref = oracle.prefill(host(x.q_out), host(x.kc), host(x.vc), tables.cpu().numpy(),
                         np.array(lens, np.int32), start.cpu().numpy(), scale, dtype)
    assert np.abs(out.double().cpu().numpy() - ref).max() <= TOL[dtype]
    for step in range(4):
        lens = [L + 1 for L in lens]
        y = Tokens(n, hq, hkv, d, dtype, seed=20 + step)
        y.cs, y.qw, y.kw, y.kc, y.vc = x.cs, x.qw, x.kw, x.kc, x.vc
        y.pos = torch.tensor([L - 1 for L in lens]).int().cuda()
        y.slots = torch.stack([tables[s, (L - 1) // 16].long() * 16 + (L - 1) % 16
                               for s, L in enumerate(lens)])
        tl = torch.tensor(lens).int().cuda()
        out = torch.empty_like(y.q_out)
        if step % 2:
            pa.qk_norm_rope(y.q, y.k, y.q, y.k, y.pos, y.cs, q_norm=y.qw, k_norm=y.kw, eps=EPS)
            pa.decode_append(out, y.q, y.kc, y.vc, tables, tl, y.k, y.v, y.slots, scale)
            q = y.q
        else:
            y.append(pa)
            pa.decode(out, y.q_out, y.kc, y.vc, tables, tl, scale)
            q = y.q_out
        torch.cuda.synchronize()
        ref = oracle.decode(host(q), host(y.kc), host(y.vc), tables.cpu().numpy(),
                            np.array(lens, np.int32), scale, dtype)
        assert np.abs(out.double().cpu().numpy() - ref).max() <= TOL[dtype]
        assert pa.get_device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hkv,maps,rot,norm,fused", [(9001, 10, 2, 1, 96, "k", False),
                                                          (8003, 24, 8, 2, 48, "qk", True)])
def test_append_through_the_rings_128_channels_f16(pa, t, hq, hkv, maps, rot, norm, fused, inter):
    # rows go through the rings above three units of (at most four) rounds a resident warp
    d = 128
    rounds = -(-(hq + 2 * hkv) * maps // (512 * maps // d))
    assert t * -(-rounds // 4) > 3 * 16 * torch.cuda.get_device_properties(0).multi_processor_count
    x = Tokens(t, hq, hkv, d, "f16", maps, rot, norm, fused, seed=t)
    x.slots[5], x.pos[t - 2] = -1, -3
    x.check(pa, lambda: x.append(pa, inter), inter, skipped=[5, t - 2])
    assert pa.get_device_error() == 0
