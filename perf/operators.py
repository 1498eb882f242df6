"""The token-preparation and differential-attention operators, measured.

Four operators over the paged KV pool, each in its plain form (elementary torch
operations in 32 bits) and, where ``own`` is true, as the call a serving
program makes:

  rope_and_cache  rotate (and optionally normalise) q and k, write k and v into
                  their pool slots
  qk_norm_rope    normalise and rotate q and k of new tokens, no pool
  diff_decode     differential attention of one query token per sequence over
                  the pool
  diff_prefill    the same for prompt chunks, causal
"""
import math
import statistics

import torch

own = False

BLOCK = 16
EPS = 1e-6
THETA = 10000.0
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token of a small model: all latency
        dict(name="append 1 token", op="rope_and_cache", dtype="f16", tokens=1, hq=8, hkv=8, d=64,
             maps=1, rot=64, inter=False, norm=False, table=4096, chunk=0, fused=False),
        # a decode step of the batch-128 GQA workload, q, k, v being slices of
        # one projection's output
        dict(name="append decode step", op="rope_and_cache", dtype="bf16", tokens=128, hq=32,
             hkv=8, d=128, maps=1, rot=128, inter=False, norm=True, table=4096, chunk=0,
             fused=True),
        # 16 prompt chunks of 2048 tokens in one step
        dict(name="append prompt chunks", op="rope_and_cache", dtype="bf16", tokens=32768, hq=32,
             hkv=8, d=128, maps=1, rot=128, inter=False, norm=True, table=16384, chunk=2048,
             fused=True),
        # a decode step of the MHA workload, whose decode appends the tokens itself
        dict(name="norm decode step", op="qk_norm_rope", dtype="f16", tokens=64, hq=32, hkv=32,
             d=128, maps=1, rot=128, inter=True, norm=True, table=2048, chunk=0, fused=False),
        # two keys a head for differential attention, odd token count
        dict(name="norm two maps", op="qk_norm_rope", dtype="bf16", tokens=777, hq=32, hkv=8,
             d=128, maps=2, rot=64, inter=False, norm=True, table=8192, chunk=0, fused=True),
        # prompt chunks, partial rotation
        dict(name="norm prompt chunks", op="qk_norm_rope", dtype="f16", tokens=16384, hq=40,
             hkv=8, d=128, maps=1, rot=64, inter=False, norm=True, table=16384, chunk=1024,
             fused=True),
        # four short sequences: latency
        dict(name="diff decode short", op="diff_decode", dtype="f16", seqs=4, hq=8, hkv=8, d=64,
             lens="uniform", lo=1, hi=100, norm=True),
        # the batch-128 GQA workload's lengths
        dict(name="diff decode batch", op="diff_decode", dtype="bf16", seqs=128, hq=32, hkv=8,
             d=128, lens="lognormal", lo=16, hi=4096, norm=True),
        # long contexts, few sequences
        dict(name="diff decode long", op="diff_decode", dtype="bf16", seqs=4, hq=32, hkv=8, d=128,
             lens="uniform", lo=32768, hi=131072, norm=True),
        # two ragged chunks of short prompts
        dict(name="diff prefill short", op="diff_prefill", dtype="f16", seqs=2, hq=8, hkv=2, d=64,
             clo=5, chi=70, lo=70, hi=150, norm=True),
        # 512-token chunks over contexts of 0.5K to 4K
        dict(name="diff prefill chunks", op="diff_prefill", dtype="bf16", seqs=8, hq=32, hkv=8,
             d=128, clo=512, chi=512, lo=512, hi=4096, norm=True),
        # long prompts: 2048-token chunks at 16K
        dict(name="diff prefill long", op="diff_prefill", dtype="bf16", seqs=2, hq=32, hkv=8,
             d=128, clo=2048, chi=2048, lo=16384, hi=16384, norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_and_cache", "qk_norm_rope", "diff_decode", "diff_prefill"])
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]))
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    c.update(d=d, hkv=hkv)
    if op in ("rope_and_cache", "qk_norm_rope"):
        maps = rng.choice([1, 1, 2])
        c.update(hq=hkv * rng.choice([1, 2, 3, 4, 5, 8]) if hkv <= 8 else hkv,
                 maps=maps, inter=rng.random() < 0.4, norm=rng.random() < 0.7,
                 rot=16 * rng.randint(1, d // maps // 16), table=_log(rng, 1024, 131072),
                 fused=rng.random() < 0.5, chunk=0)
        # no more bytes than the largest listed case moves
        most = 32768 * 48 * 128 // ((c["hq"] + 2 * hkv) * d)
        c["tokens"] = _log(rng, 1, min(most, 65536))
        if rng.random() < 0.4:
            c["chunk"] = min(_log(rng, 16, 2048), c["table"], c["tokens"])
        return c
    c.update(norm=rng.random() < 0.8, hq=hkv * rng.randint(1, 8))
    if op == "diff_decode":
        # K/V bytes, padded for the plain form, below the long case's
        tokens = 4 * 131072 * 8 * 128 // (hkv * d)
        c["lens"] = rng.choice(["uniform", "lognormal"])
        c["seqs"] = _log(rng, 1, 200)
        c["hi"] = _log(rng, 2, min(131072, max(2, tokens // (2 * c["seqs"]))))
        c["lo"] = rng.randint(0, c["hi"] // 2)
        return c
    c["seqs"] = rng.randint(1, 8)
    while True:
        c["chi"] = _log(rng, 1, 2048)
        c["clo"] = rng.randint(1, c["chi"])
        c["hi"] = _log(rng, c["chi"], 16384) if c["chi"] < 16384 else 16384
        c["lo"] = rng.randint(c["chi"], c["hi"])
        if c["seqs"] * c["chi"] * c["hi"] * c["hq"] * d <= 2048 * 16384 * 32 * 128:
            return c


def _spread(kind, n, lo, hi):
    """n whole numbers over [lo, hi], the same for every seed but for their order."""
    if n == 1:
        return [hi]
    if kind == "lognormal":
        q = [math.exp(math.log(max(1, hi) / 6.8) + statistics.NormalDist().inv_cdf((i + 0.5) / n))
             for i in range(n)]
        return [min(hi, max(lo, int(round(x)))) for x in q]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(c):
    return _spread(c.get("lens", "uniform"), c["seqs"], c["lo"], c["hi"])


def _chunks(c):
    return _spread("uniform", c["seqs"], c["clo"], c["chi"])


def work(c):
    d = c["d"]
    if c["op"] in ("rope_and_cache", "qk_norm_rope"):
        t, q, k = c["tokens"], c["hq"] * d, c["hkv"] * d
        rows = min(c["chunk"] or c["table"], t, c["table"]) * c["rot"] * 4
        if c["op"] == "rope_and_cache":
            return {"bytes": t * (2 * q + 4 * k) * 2 + rows + 12 * t, "flops": t * (q + k) * 3}
        return {"bytes": t * (2 * q + 2 * k) * 2 + rows + 4 * t, "flops": t * (q + k) * 6}
    lens = _lens(c)
    if c["op"] == "diff_decode":
        kv = sum(lens) * c["hkv"] * d * 4
        return {"bytes": kv + c["seqs"] * c["hq"] * d * 4, "flops": sum(lens) * c["hq"] * 6 * d}
    chunks = _chunks(c)
    # as many pairs as the chunks' order over the lengths gives on average
    mean_len = sum(lens) / len(lens)
    pairs = sum(n * mean_len - n * (n - 1) / 2 for n in chunks)
    return {"bytes": sum(lens) * c["hkv"] * d * 4 + sum(chunks) * c["hq"] * d * 4,
            "flops": pairs * c["hq"] * 6 * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _angles(table, rot, dev):
    pos = torch.arange(table, device=dev, dtype=torch.float64)
    inv = THETA ** (-2.0 * torch.arange(rot // 2, device=dev, dtype=torch.float64) / rot)
    return pos[:, None] * inv


def _rows(g, shape, dt, dev, gain=1.0):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(gain).to(dt)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt, d, hq, hkv = TORCH[c["dtype"]], c["d"], c["hq"], c["hkv"]
    s = dict(case=c)
    if c["op"] in ("rope_and_cache", "qk_norm_rope"):
        t = c["tokens"]
        if c["fused"]:
            # one projection's output, q | k | v per token
            qkv = _rows(g, (t, (hq + 2 * hkv) * d), dt, dev)
            s["q"] = qkv[:, :hq * d].view(t, hq, d)
            s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
            s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        else:
            s["q"], s["k"], s["v"] = (_rows(g, (t, h, d), dt, dev) for h in (hq, hkv, hkv))
        a = _angles(c["table"], c["rot"], dev)
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        if c["chunk"]:
            i = torch.arange(t, device=dev)
            s["positions"] = (i % c["chunk"] + (c["table"] - c["chunk"])).int()
        else:
            s["positions"] = torch.randint(0, c["table"], (t,), generator=g, device=dev).int()
        s["q_norm"] = s["k_norm"] = None
        if c["norm"]:
            # learned weights of these norms lie around one
            s["q_norm"], s["k_norm"] = (
                (1 + 0.2 * torch.randn(d // c["maps"], generator=g, device=dev)).to(dt)
                for _ in range(2))
        s["q_out"] = torch.zeros(t, hq, d, device=dev, dtype=dt)
        if c["op"] == "qk_norm_rope":
            s["k_out"] = torch.zeros(t, hkv, d, device=dev, dtype=dt)
            return s
        blocks = (t + BLOCK - 1) // BLOCK if c["chunk"] else t
        nb = blocks + blocks // 4 + 1
        order = torch.randperm(nb, generator=g, device=dev)[:blocks]
        i = torch.arange(t, device=dev)
        if c["chunk"]:
            s["slots"] = order[i // BLOCK] * BLOCK + i % BLOCK
        else:
            # one token of each of many sequences, anywhere in its last block
            s["slots"] = order * BLOCK + torch.randint(0, BLOCK, (t,), generator=g, device=dev)
        s["k_cache"] = _rows(g, (nb, hkv, BLOCK, d), dt, dev)
        s["v_cache"] = _rows(g, (nb, hkv, BLOCK, d), dt, dev)
        return s
    n, lens = c["seqs"], _lens(c)
    perm = torch.randperm(n, generator=g, device=dev).tolist()
    lens = [lens[i] for i in perm]
    mb = max(1, (max(lens) + BLOCK - 1) // BLOCK)
    used = [(x + BLOCK - 1) // BLOCK for x in lens]
    nb = sum(used) + sum(used) // 4 + 1
    order = torch.randperm(nb, generator=g, device=dev)[:sum(used)].int()
    need = torch.tensor(used, device=dev)
    at = torch.arange(mb, device=dev)[None]
    first = (need.cumsum(0) - need)[:, None]
    live = at < need[:, None]
    tables = torch.full((n, mb), -1, device=dev, dtype=torch.int32)
    if sum(used):
        picked = order[(first + at).clamp(max=sum(used) - 1)]
        tables = torch.where(live, picked, tables)
    s["tables"] = tables.contiguous()
    s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    s["k_cache"] = _rows(g, (nb, hkv, BLOCK, d), dt, dev)
    s["v_cache"] = _rows(g, (nb, hkv, BLOCK, d), dt, dev)
    s["scale"] = (d // 2) ** -0.5
    # trained weights of the difference lie between 0.2 and 0.8
    s["lam"] = 0.2 + 0.6 * torch.rand(hq, generator=g, device=dev)
    s["norm_w"] = ((1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
                   if c["norm"] else None)
    s["out_scale"] = 0.2 if c["norm"] else 1.0
    if c["op"] == "diff_decode":
        rows = n
    else:
        chunks = _chunks(c)
        start = [0]
        for x in chunks:
            start.append(start[-1] + x)
        s["start"] = torch.tensor(start, device=dev, dtype=torch.int32)
        s["longest"] = max(chunks)
        rows = start[-1]
    # normalised queries and keys leave scores a standard deviation of about two
    s["q"] = _rows(g, (rows, hq, d), dt, dev, 2.0)
    s["out"] = torch.zeros(rows, hq, d, device=dev, dtype=dt)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _norm_rope(x, w, cos, sin, c):
    """x [tokens, heads, d] in 32 bits out, normalised and rotated per segment."""
    t, h, d = x.shape
    seg, rot = d // c["maps"], c["rot"]
    y = x.float().reshape(t, h * c["maps"], seg)
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    r = y[..., :rot]
    if c["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if c["inter"] else torch.cat([a, b], -1)
    return torch.cat([r, y[..., rot:]], -1).reshape(t, h, d)


def _prepared(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, None, :c["rot"] // 2], cs[:, None, c["rot"] // 2:]
    s["q_out"].copy_(_norm_rope(s["q"], s["q_norm"], cos, sin, c))
    return _norm_rope(s["k"], s["k_norm"], cos, sin, c)


def _gathered(pool, tables):
    """Each sequence's rows through its table: [n, hkv, tokens, d] in 32 bits."""
    x = pool[tables.long().clamp(min=0)]
    n, mb, hkv, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, mb * b, d).float()


def _softmax_pv(q, k, v, seen, scale):
    """q [n, hkv, rows, d/2], k [n, hkv, t, d/2], v [n, hkv, t, d]; seen masks keys."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    return torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-38)


def _difference(s, q, seen, live):
    """q [n, hkv, rows, g, d] in 32 bits, seen [n, 1, rows * g, t] -> [n, hkv, rows, g, d]."""
    c = s["case"]
    n, hkv, rows, g, d = q.shape
    k, v = _gathered(s["k_cache"], s["tables"]), _gathered(s["v_cache"], s["tables"])
    v = v.masked_fill(~live, 0.0)
    q = q.reshape(n, hkv, rows * g, d)
    h = d // 2
    o1 = _softmax_pv(q[..., :h], k[..., :h], v, seen, s["scale"])
    o2 = _softmax_pv(q[..., h:], k[..., h:], v, seen, s["scale"])
    y = (o1.reshape(n, hkv, rows, g, d)
         - s["lam"].reshape(1, hkv, 1, g, 1) * o2.reshape(n, hkv, rows, g, d))
    if c["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["norm_w"].float()
    return y * s["out_scale"]


def _plain(s):
    c = s["case"]
    if c["op"] == "qk_norm_rope":
        s["k_out"].copy_(_prepared(s))
        return s["q_out"], s["k_out"]
    if c["op"] == "rope_and_cache":
        k = _prepared(s)
        blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
        s["k_cache"][blk, :, off] = k.to(s["k_cache"].dtype)
        s["v_cache"][blk, :, off] = s["v"]
        return s["q_out"], s["k_cache"], s["v_cache"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    at = torch.arange(s["tables"].shape[1] * BLOCK, device=s["q"].device)
    lens = s["lens"].long()
    live = (at[None] < lens[:, None])[:, None, :, None]
    n = lens.shape[0]
    if c["op"] == "diff_decode":
        q = s["q"].float().reshape(n, hkv, 1, g, d)
        y = _difference(s, q, live.transpose(-1, -2), live)
        s["out"].copy_(y.reshape(n, hq, d))
        return s["out"]
    start = s["start"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(s["longest"], device=at.device)
    rows = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().reshape(n, s["longest"], hkv, g, d).permute(0, 2, 1, 3, 4)
    pos = (lens - count)[:, None] + i
    seen = (at[None, None] <= pos[..., None]) & (at[None, None] < lens[:, None, None])
    seen = seen[:, None, :, None].expand(n, 1, s["longest"], g, at.shape[0])
    y = _difference(s, q, seen.reshape(n, 1, s["longest"] * g, at.shape[0]), live)
    # back to the packed rows
    r = torch.arange(s["q"].shape[0], device=at.device)
    seq = torch.searchsorted(start[1:].contiguous(), r, right=True)
    s["out"].copy_(y[seq, :, r - start[seq]].reshape(-1, hq, d))
    return s["out"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if not own:
        return _plain(s)
    import paged_kv_cache_260_gb300 as pa
    c = s["case"]
    if c["op"] == "rope_and_cache":
        pa.rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                          s["slots"], s["positions"], s["cos_sin"], q_norm=s["q_norm"],
                          k_norm=s["k_norm"], eps=EPS, interleaved=c["inter"],
                          num_maps=c["maps"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if c["op"] == "qk_norm_rope":
        pa.qk_norm_rope(s["q_out"], s["k_out"], s["q"], s["k"], s["positions"], s["cos_sin"],
                        q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, interleaved=c["inter"],
                        num_maps=c["maps"])
        return s["q_out"], s["k_out"]
    if c["op"] == "diff_decode":
        if "workspace" not in s:
            s["workspace"] = pa.diff_decode_workspace_for(s["q"], s["k_cache"], s["tables"])
        return pa.diff_decode(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"],
                              s["lens"], s["lam"], s["scale"], norm_weight=s["norm_w"], eps=EPS,
                              out_scale=s["out_scale"], workspace=s["workspace"])
    if "workspace" not in s:
        s["workspace"] = pa.diff_prefill_workspace_for(s["q"], s["k_cache"], s["lens"],
                                                       s["longest"])
    return pa.diff_prefill(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                           s["start"], s["longest"], s["lam"], s["scale"],
                           norm_weight=s["norm_w"], eps=EPS, out_scale=s["out_scale"],
                           workspace=s["workspace"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(x, w, ang, c):
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    seg, rot = c["d"] // c["maps"], c["rot"]
    for m in range(c["maps"]):
        y = x[..., m * seg:(m + 1) * seg].double()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / seg + EPS).sqrt() * w.double()
        z = y.clone()
        i = torch.arange(rot // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rot // 2)
        # the pair as a complex number, turned by its angle
        turned = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(ang), ang)
        z[..., a], z[..., b] = turned.real, turned.imag
        out[..., m * seg:(m + 1) * seg] = z
    return out


def _exact_rows(s, c, seq, pos, q):
    """q [rows, hq, d] at positions pos of one sequence."""
    g, d = c["hq"] // c["hkv"], c["d"]
    t = int(pos.max()) + 1 if pos.numel() else 0
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    if t == 0:
        return out
    blocks = s["tables"][seq, :(t + BLOCK - 1) // BLOCK].long()
    hidden = torch.arange(t, device=q.device)[None] > pos[:, None]
    for h in range(c["hkv"]):
        k = s["k_cache"][blocks, h].reshape(-1, d)[:t].double()
        v = s["v_cache"][blocks, h].reshape(-1, d)[:t].double()
        for j in range(h * g, h * g + g):
            y = torch.zeros(q.shape[0], d, dtype=torch.float64, device=q.device)
            for part, sign in ((slice(0, d // 2), 1.0), (slice(d // 2, d), -s["lam"][j].double())):
                x = q[:, j, part].double() @ k[:, part].T * s["scale"]
                y += sign * (torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v)
            if s["norm_w"] is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * s["norm_w"].double()
            out[:, j] = y * s["out_scale"]
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("rope_and_cache", "qk_norm_rope"):
        ang = _angles(c["table"], c["rot"], s["q"].device)[s["positions"].long()][:, None]
        q, k = (_exact_rope(s[x], s[x + "_norm"], ang, c) for x in "qk")
        if c["op"] == "qk_norm_rope":
            return q, k
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
        for h in range(c["hkv"]):
            kc[blk, h, off] = k[:, h]
            vc[blk, h, off] = s["v"][:, h].double()
        return q, kc, vc
    lens = s["lens"].tolist()
    out = []
    if c["op"] == "diff_decode":
        for i, n in enumerate(lens):
            pos = torch.tensor([n - 1], device=s["q"].device)
            out.append(_exact_rows(s, c, i, pos, s["q"][i:i + 1]))
        return torch.cat(out)
    start = s["start"].tolist()
    for i, n in enumerate(lens):
        rows = start[i + 1] - start[i]
        pos = torch.arange(n - rows, n, device=s["q"].device)
        out.append(_exact_rows(s, c, i, pos, s["q"][start[i]:start[i + 1]]))
    return torch.cat(out)
