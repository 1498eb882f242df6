"""Sparse attention over selected blocks, and eviction by attention weight, measured.

Six operators over the paged KV pool, each in its plain form (elementary torch
operations) and, where ``own`` is true, as the call a serving program makes:

  block_bounds   per block and kv head, the least and greatest key of each channel
  select_blocks  per sequence and kv head, the blocks whose bounds promise the
                 largest scores for the new token's queries
  sparse_decode  decode attention over the selected blocks
  decode_mass    decode attention that adds each token's softmax weights to its
                 accumulated weight ("mass")
  prefill_mass   the weights that the queries of a prompt chunk give every token
  evict          a sequence shortened to its heaviest tokens, in place
"""
import math
import statistics

import torch

own = False

BLOCK = 16
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # after a decode step: the block of each sequence's newest token
        dict(name="bounds decode step", op="block_bounds", dtype="bf16", seqs=128, hkv=8, d=128,
             lens="lognormal", lo=16, hi=4096, step=True),
        # after prompts of 16K tokens: every block
        dict(name="bounds prompts", op="block_bounds", dtype="bf16", seqs=16, hkv=8, d=128,
             lens="uniform", lo=16384, hi=16384, step=False),
        # a small model, four sequences: latency
        dict(name="select few", op="select_blocks", dtype="f16", seqs=4, hq=8, hkv=8, d=64,
             lens="uniform", lo=100, hi=1024, keep=16, first=1, last=1),
        # contexts of 32K to 131K
        dict(name="select long", op="select_blocks", dtype="bf16", seqs=4, hq=32, hkv=8, d=128,
             lens="uniform", lo=32768, hi=131072, keep=256, first=4, last=8),
        # attention over such selections: the small model's, and 1024 tokens for each of 128
        dict(name="sparse decode few", op="sparse_decode", dtype="f16", seqs=4, hq=8, hkv=8, d=64,
             lens="uniform", lo=100, hi=1024, keep=16),
        dict(name="sparse decode batch", op="sparse_decode", dtype="bf16", seqs=128, hq=32, hkv=8,
             d=128, lens="uniform", lo=512, hi=4096, keep=64),
        # a decode step that keeps account: the batch-128 workload's lengths
        dict(name="mass decode batch", op="decode_mass", dtype="bf16", seqs=128, hq=32, hkv=8,
             d=128, lens="lognormal", lo=16, hi=4096, decay=1.0),
        # four short sequences, old weights fading
        dict(name="mass decode short", op="decode_mass", dtype="f16", seqs=4, hq=8, hkv=8, d=64,
             lens="uniform", lo=1, hi=100, decay=0.98),
        # two ragged chunks of short prompts
        dict(name="mass prefill short", op="prefill_mass", dtype="f16", seqs=2, hq=8, hkv=2, d=64,
             clo=5, chi=70, lo=70, hi=150, decay=1.0),
        # the last 64 queries of 16K prompts say what is kept of them
        dict(name="mass prefill window", op="prefill_mass", dtype="bf16", seqs=8, hq=32, hkv=8,
             d=128, clo=64, chi=64, lo=16384, hi=16384, decay=0.0),
        # a batch that grows by one block and gives it back
        dict(name="evict block", op="evict", dtype="bf16", seqs=128, hkv=8, d=128, lens="uniform",
             lo=1040, hi=1040, new=1024, first=4, last=32),
        # prompts cut down to 2048 tokens
        dict(name="evict prompts", op="evict", dtype="bf16", seqs=8, hkv=8, d=128, lens="uniform",
             lo=8192, hi=32768, new=2048, first=4, last=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block_bounds", "select_blocks", "sparse_decode", "decode_mass",
                     "prefill_mass", "evict"])
    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), d=d, hkv=hkv)
    if op != "block_bounds" and op != "evict":
        c["hq"] = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16] if hkv <= 4 else [1, 2, 4, 5, 8])
    if op == "prefill_mass":
        c.update(seqs=rng.randint(1, 8), decay=rng.choice([0.0, 0.9, 1.0]))
        while True:
            c["chi"] = _log(rng, 1, 2048)
            c["clo"] = rng.randint(1, c["chi"])
            c["hi"] = _log(rng, c["chi"], 32768)
            c["lo"] = rng.randint(c["chi"], c["hi"])
            if c["seqs"] * c["chi"] * c["hi"] * c["hq"] * d <= 8 * 64 * 16384 * 32 * 128:
                return c
    # tokens of all sequences: no more K/V than the largest listed cases have
    tokens = 16 * 16384 * 8 * 128 // (hkv * d)
    c["lens"] = rng.choice(["uniform", "lognormal"])
    c["seqs"] = _log(rng, 1, 200)
    c["hi"] = _log(rng, 2, min(131072, max(2, tokens // (2 * c["seqs"]))))
    c["lo"] = rng.randint(0, c["hi"] // 2)
    if op == "block_bounds":
        c["step"] = rng.random() < 0.5
        c["lo"] = max(c["lo"], int(c["step"]))          # a step gives every sequence a token
    elif op in ("select_blocks", "sparse_decode"):
        c["keep"] = _log(rng, 1, 512)
        if op == "sparse_decode":
            c["keep"] = min(c["keep"], max(1, 128 * 64 * 8 * 128 // (c["seqs"] * hkv * d)))
        else:
            c["last"] = rng.randint(1, min(8, c["keep"]))
            c["first"] = rng.randint(0, min(4, c["keep"] - c["last"]))
    elif op == "decode_mass":
        c["decay"] = rng.choice([0.0, 0.9, 1.0])
    else:
        c["new"] = _log(rng, 1, c["hi"] - 1)
        c["last"] = rng.randint(0, min(c["new"], 128))
        c["first"] = rng.randint(0, 4)
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


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(c):
    d, hkv, lens = c["d"], c["hkv"], _lens(c)
    hq, n = c.get("hq", 0), c["seqs"]
    blocks = sum(_blocks(x) for x in lens)
    if c["op"] == "block_bounds":
        if c["step"]:
            keys, blocks = sum((x - 1) % BLOCK + 1 for x in lens), n
        else:
            keys = sum(lens)
        return {"bytes": keys * hkv * d * 2 + blocks * hkv * (4 * d) + 4 * blocks,
                "flops": keys * hkv * 2 * d}
    if c["op"] == "select_blocks":
        # sequences that fit in the selection need no scores
        scored = sum(_blocks(x) for x in lens if _blocks(x) > c["keep"])
        return {"bytes": scored * hkv * 4 * d + n * hq * d * 2 + 4 * blocks
                + n * hkv * (c["keep"] + 1) * 4, "flops": scored * hq * 4 * d}
    if c["op"] == "sparse_decode":
        tokens = sum(x if _blocks(x) <= c["keep"] else
                     (c["keep"] - 1) * BLOCK + (x - 1) % BLOCK + 1 for x in lens)
        return {"bytes": tokens * hkv * d * 4 + n * hq * d * 4, "flops": tokens * hq * 4 * d}
    if c["op"] == "decode_mass":
        old = 4 if c["decay"] else 0
        return {"bytes": sum(lens) * hkv * (d * 4 + 4 + old) + n * hq * d * 4,
                "flops": sum(lens) * hq * 4 * d}
    if c["op"] == "prefill_mass":
        chunks, mean_len = _chunks(c), sum(lens) / n
        old = 4 if c["decay"] else 0
        pairs = sum(m * mean_len - m * (m - 1) / 2 for m in chunks)
        return {"bytes": sum(lens) * hkv * (2 * d + 4 + old) + sum(chunks) * hq * d * 2,
                "flops": pairs * hq * 2 * d}
    moved = 0.0
    for x in lens:
        if x <= c["new"]:
            continue
        last = min(c["last"], c["new"])
        first = min(c["first"], c["new"] - last)
        heavy = c["new"] - last - first
        # as many of the heaviest lie past the new end as of any
        moved += last + heavy * (1 - heavy / (x - last - first))
    return {"bytes": sum(x for x in lens if x > c["new"]) * hkv * 4
            + moved * hkv * (8 * d + 8) + 8 * n, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(g, shape, dt, dev, gain=1.0):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(gain).to(dt)


def _keys(g, nb, hkv, d, dt, dev):
    """Keys as rotated ones are spread: each block's lie around a centre of its own."""
    k = torch.randn(nb, hkv, BLOCK, d, generator=g, device=dev, dtype=torch.float32).mul_(0.8)
    return k.add_(torch.randn(nb, hkv, 1, d, generator=g, device=dev), alpha=0.6).to(dt)


def _with_bounds(old, k, tables, lens):
    """The pool's bounds with those of every block of these sequences in place."""
    nb = k.shape[0]
    at = torch.arange(tables.shape[1], device=k.device)
    live = (lens[:, None] - BLOCK * at[None]).clamp(0, BLOCK).long()
    # tokens that each block holds; what no table names goes to a spare entry
    held = torch.zeros(nb + 1, device=k.device, dtype=torch.long)
    held.scatter_(0, torch.where(live > 0, tables, nb).long().flatten(), live.flatten())
    held = held[:nb]
    dead = (torch.arange(BLOCK, device=k.device)[None] >= held[:, None])[:, None, :, None]
    least = k.masked_fill(dead, math.inf).amin(2)
    most = k.masked_fill(dead, -math.inf).amax(2)
    new = torch.stack([least, most], 2)
    return torch.where((held > 0)[:, None, None, None], new, old)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt, d, hkv, n = TORCH[c["dtype"]], c["d"], c["hkv"], c["seqs"]
    hq = c.get("hq", hkv)
    s, lens = dict(case=c), _lens(c)
    perm = torch.randperm(n, generator=g, device=dev).tolist()
    lens = [lens[i] for i in perm]
    mb = max(1, _blocks(max(lens)))
    used = [_blocks(x) for x in lens]
    total = sum(used)
    nb = total + total // 4 + 1
    order = torch.randperm(nb, generator=g, device=dev)[:total].int()
    need = torch.tensor(used, device=dev)
    at = torch.arange(mb, device=dev)[None]
    first = (need.cumsum(0) - need)[:, None]
    live = at < need[:, None]
    tables = torch.full((n, mb), -1, device=dev, dtype=torch.int32)
    if total:
        tables = torch.where(live, order[(first + at).clamp(max=total - 1)], tables)
    s["tables"] = tables.contiguous()
    s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    s["k_cache"] = _keys(g, nb, hkv, d, dt, dev)
    s["scale"] = d ** -0.5
    # normalised queries and keys leave scores a standard deviation of about two
    rows, op = n, c["op"]
    if op == "prefill_mass":
        start = [0]
        for x in _chunks(c):
            start.append(start[-1] + x)
        s["start"] = torch.tensor(start, device=dev, dtype=torch.int32)
        s["longest"], rows = max(_chunks(c)), start[-1]
    if op != "block_bounds" and op != "evict":
        s["q"] = _rows(g, (rows, hq, d), dt, dev, 2.0)
    if op == "block_bounds":
        s["starts"] = s["lens"] - 1 if c["step"] else None
        # what an earlier use of the blocks left
        s["bounds"] = torch.zeros(nb, hkv, 2, d, device=dev, dtype=dt)
    elif op == "select_blocks":
        zero = torch.zeros(nb, hkv, 2, d, device=dev, dtype=dt)
        s["bounds"] = _with_bounds(zero, s["k_cache"], s["tables"], s["lens"])
        del s["k_cache"]
        s["tiles"] = torch.zeros(n, hkv, c["keep"], device=dev, dtype=torch.int32)
        s["tile_lens"] = torch.zeros(n, hkv, device=dev, dtype=torch.int32)
    elif op == "sparse_decode":
        s["v_cache"] = _rows(g, (nb, hkv, BLOCK, d), dt, dev)
        # as select_blocks leaves them: some blocks of each head, the last one among them
        keep = c["keep"]
        rank = torch.rand(n, hkv, mb, generator=g, device=dev)
        rank = rank.masked_fill(~live[:, None], 2.0)
        rank = rank.masked_fill((at == need[:, None] - 1)[:, None], -1.0)
        top = rank.argsort(-1)[..., :keep]
        none = torch.arange(top.shape[-1], device=dev) >= need[:, None, None]
        top = top.masked_fill(none, mb).sort(-1).values
        heads = torch.arange(hkv, device=dev)[None, :, None]
        seq = torch.arange(n, device=dev)[:, None, None]
        tiles = s["tables"][seq, top.clamp(max=mb - 1)] * hkv + heads
        s["tiles"] = torch.full((n, hkv, keep), -1, device=dev, dtype=torch.int32)
        s["tiles"][..., :top.shape[-1]] = tiles.masked_fill(top == mb, -1).int()
        count = need.clamp(max=keep)
        s["tile_lens"] = torch.where(need > 0, s["lens"] - BLOCK * (need - count), 0)
        s["tile_lens"] = s["tile_lens"][:, None].expand(n, hkv).int().contiguous()
        s["out"] = torch.zeros(n, hq, d, device=dev, dtype=dt)
    else:
        # the weight that earlier steps gave: few tokens have most of it
        mass = torch.randn(n, hkv, mb * BLOCK, generator=g, device=dev).mul_(2.0).exp_()
        s["mass"] = mass / mass.sum(-1, keepdim=True) * 100.0
        if op == "decode_mass":
            s["v_cache"] = _rows(g, (nb, hkv, BLOCK, d), dt, dev)
            s["out"] = torch.zeros(n, hq, d, device=dev, dtype=dt)
        elif op == "evict":
            s["v_cache"] = _rows(g, (nb, hkv, BLOCK, d), dt, dev)
            s["new_lens"] = torch.full((n,), c["new"], device=dev, dtype=torch.int32)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _gathered(pool, tables):
    """Each sequence's rows through its table: [n, hkv, tokens, d] in 32 bits."""
    x = pool[tables.long().clamp(min=0)]
    n, mb, hkv, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, mb * b, d).float()


def _softmax(x, seen):
    """Weights over the last dimension; a row that sees nothing has none."""
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-38)


def _plain_bounds(s):
    k, tables, lens = s["k_cache"], s["tables"].long(), s["lens"].long()
    if s["starts"] is None:
        return s["bounds"].copy_(_with_bounds(s["bounds"], k, tables, lens))
    # one block of each sequence
    at = (lens - 1) // BLOCK
    block = tables.gather(1, at[:, None])[:, 0]
    dead = (torch.arange(BLOCK, device=k.device)[None] >= (lens - BLOCK * at)[:, None])
    dead, k = dead[:, None, :, None], k[block]
    s["bounds"][block] = torch.stack([k.masked_fill(dead, math.inf).amin(2),
                                      k.masked_fill(dead, -math.inf).amax(2)], 2)
    return s["bounds"]


def _plain_select(s):
    c = s["case"]
    n, hkv, keep = s["tiles"].shape
    tables, lens, d = s["tables"].long(), s["lens"].long(), c["d"]
    b = s["bounds"][tables.clamp(min=0)].permute(0, 2, 3, 1, 4).double()   # n, hkv, 2, mb, d
    q = s["q"].reshape(n, hkv, -1, d).double()
    score = (torch.matmul(q.clamp(min=0), b[:, :, 1].transpose(-1, -2))
             + torch.matmul(q.clamp(max=0), b[:, :, 0].transpose(-1, -2))).amax(2)
    mb = tables.shape[1]
    at = torch.arange(mb, device=q.device)[None, None]
    need = ((lens + BLOCK - 1) // BLOCK)[:, None, None]
    score = score.masked_fill((at < c["first"]) | (at >= need - c["last"]), math.inf)
    score = score.masked_fill(at >= need, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    none = torch.arange(order.shape[-1], device=q.device) >= need
    order = order.masked_fill(none, mb).sort(-1).values
    picked = tables.gather(1, order.clamp(max=mb - 1).reshape(n, -1)).reshape(order.shape)
    tiles = picked * hkv + torch.arange(hkv, device=q.device)[None, :, None]
    s["tiles"].fill_(-1)
    s["tiles"][..., :order.shape[-1]] = tiles.masked_fill(order == mb, -1).int()
    left_out = (need - keep).clamp(min=0)[..., 0]
    s["tile_lens"].copy_((lens[:, None] - BLOCK * left_out).expand(n, hkv))
    return s["tiles"], s["tile_lens"]


def _plain_sparse(s):
    n, hkv, keep = s["tiles"].shape
    d = s["q"].shape[-1]
    at = s["tiles"].long().clamp(min=0).reshape(n * hkv, keep)
    k, v = (x.reshape(-1, BLOCK, d)[at].reshape(n * hkv, keep * BLOCK, d).float()
            for x in (s["k_cache"], s["v_cache"]))
    seen = torch.arange(keep * BLOCK, device=k.device)[None] < s["tile_lens"].reshape(-1, 1)
    q = s["q"].float().reshape(n * hkv, -1, d)
    p = _softmax(torch.matmul(q, k.transpose(-1, -2)) * s["scale"], seen[:, None])
    y = torch.matmul(p, v.masked_fill(~seen[..., None], 0.0))
    s["out"].copy_(y.reshape(s["out"].shape))
    return s["out"]


def _plain_decode(s):
    c = s["case"]
    n, d, hkv = c["seqs"], c["d"], c["hkv"]
    k, v = _gathered(s["k_cache"], s["tables"]), _gathered(s["v_cache"], s["tables"])
    at = torch.arange(k.shape[2], device=k.device)[None]
    lens = s["lens"].long()[:, None]
    live = at < lens
    q = s["q"].float().reshape(n, hkv, -1, d)
    p = _softmax(torch.matmul(q, k.transpose(-1, -2)) * s["scale"], live[:, None, None])
    y = torch.matmul(p, v.masked_fill(~live[:, None, :, None], 0.0))
    s["out"].copy_(y.reshape(s["out"].shape))
    _add_mass(s, p.sum(2), live, at == lens - 1)
    return s["out"], s["mass"]


def _add_mass(s, new, live, fresh):
    """Live tokens' mass; those of this call (fresh) have none from before."""
    old = s["mass"].masked_fill(fresh[:, None], 0.0)
    decay = s["case"]["decay"]
    total = new if decay == 0.0 else old * decay + new
    s["mass"].copy_(torch.where(live[:, None], total, s["mass"]))


def _plain_prefill(s):
    c = s["case"]
    n, d, hkv, longest = c["seqs"], c["d"], c["hkv"], s["longest"]
    k = _gathered(s["k_cache"], s["tables"])
    start, lens = s["start"].long(), s["lens"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(longest, device=k.device)
    rows = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    g = c["hq"] // hkv
    q = s["q"][rows].float().reshape(n, longest, hkv, g, d).permute(0, 2, 3, 1, 4)
    at = torch.arange(k.shape[2], device=k.device)
    pos = (lens - count)[:, None] + i
    seen = (at <= pos[..., None]) & (i < count[:, None])[..., None]        # n, longest, t
    x = torch.matmul(q, k[:, :, None].transpose(-1, -2)) * s["scale"]
    p = _softmax(x, seen[:, None, None])
    live = at[None] < lens[:, None]
    _add_mass(s, p.sum((2, 3)), live, live & (at[None] >= (lens - count)[:, None]))
    return s["mass"]


def _plain_evict(s):
    c = s["case"]
    mass, lens = s["mass"], s["lens"].long()[:, None, None]
    n, hkv, w = mass.shape
    dev = mass.device
    new = torch.minimum(s["new_lens"].long()[:, None, None], lens)
    last = new.clamp(max=c["last"])
    first = (new - last).clamp(max=c["first"])
    heavy = new - last - first
    at = torch.arange(w, device=dev)[None, None]
    begin, end = first, lens - last                   # slots that compete
    m = mass.masked_fill((at < begin) | (at >= end), -math.inf)
    order = m.sort(dim=-1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(2, order, at.expand_as(order).contiguous())
    kept = (place < heavy) & (at >= begin) & (at < end)
    # the j-th kept slot past the heavy ones' end moves to the j-th hole before it
    edge = first + heavy
    hole = (at >= begin) & (at < edge) & ~kept
    mover = kept & (at >= edge)
    spare = w
    j_hole = torch.where(hole, hole.long().cumsum(-1) - 1, spare)
    j_move = torch.where(mover, mover.long().cumsum(-1) - 1, spare)
    to = torch.zeros(n, hkv, w + 1, device=dev, dtype=torch.long)
    to.scatter_(2, j_hole, at.expand(n, hkv, w))
    dst = torch.where(mover, to.gather(2, j_move), at)
    dst = torch.where((at >= end) & (at < lens), at - (lens - new), dst)
    moves = mover | ((at >= end) & (at < lens))
    src = torch.arange(w + 1, device=dev).expand(n, hkv, w + 1).contiguous()
    src.scatter_(2, torch.where(moves & (new < lens), dst, spare), at.expand(n, hkv, w))
    src = src[..., :w]
    mass.copy_(mass.gather(2, src))
    # the same for the pool's rows, each head its own; unused slots go to a spare row
    nb = s["k_cache"].shape[0]
    block = s["tables"].long().repeat_interleave(BLOCK, 1)[:, None]
    row = block * BLOCK + at % BLOCK                              # n, 1, w
    from_row = row.expand(n, hkv, w).gather(2, src)
    to_row = torch.where(at < lens, row, nb * BLOCK).expand(n, hkv, w)
    heads = torch.arange(hkv, device=dev)[None, :, None].expand(n, hkv, w)
    whole = torch.arange(nb * BLOCK + 1, device=dev)[:, None].repeat(1, hkv)
    whole[to_row, heads] = torch.where(at < lens, from_row, nb * BLOCK)
    whole = whole[:-1]
    for pool in (s["k_cache"], s["v_cache"]):
        x = pool.transpose(1, 2).reshape(nb * BLOCK, hkv, -1)
        x = x[whole, torch.arange(hkv, device=dev)[None]]
        pool.copy_(x.reshape(nb, BLOCK, hkv, -1).transpose(1, 2))
    return s["k_cache"], s["v_cache"], mass


PLAIN = {"block_bounds": _plain_bounds, "select_blocks": _plain_select,
         "sparse_decode": _plain_sparse, "decode_mass": _plain_decode,
         "prefill_mass": _plain_prefill, "evict": _plain_evict}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if not own:
        return PLAIN[c["op"]](s)
    import paged_kv_cache_260_gb300 as pa
    if c["op"] == "block_bounds":
        return pa.block_bounds(s["bounds"], s["k_cache"], s["tables"], s["lens"],
                               starts=s["starts"])
    if c["op"] == "select_blocks":
        if "workspace" not in s:
            s["workspace"] = pa.select_blocks_workspace_for(s["q"], s["bounds"], s["tables"])
        return pa.select_blocks(s["tiles"], s["tile_lens"], s["q"], s["bounds"], s["tables"],
                                s["lens"], keep_first=c["first"], keep_last=c["last"],
                                workspace=s["workspace"])
    if c["op"] == "sparse_decode":
        if "workspace" not in s:
            s["workspace"] = pa.sparse_decode_workspace_for(s["q"], s["k_cache"], s["tiles"])
        return pa.sparse_decode(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tiles"],
                                s["tile_lens"], s["scale"], workspace=s["workspace"])
    if c["op"] == "decode_mass":
        if "workspace" not in s:
            s["workspace"] = pa.decode_mass_workspace_for(s["q"], s["k_cache"], s["tables"])
        return pa.decode_mass(s["out"], s["mass"], s["q"], s["k_cache"], s["v_cache"],
                              s["tables"], s["lens"], s["scale"], decay=c["decay"],
                              workspace=s["workspace"])
    if c["op"] == "prefill_mass":
        if "workspace" not in s:
            s["workspace"] = pa.prefill_mass_workspace_for(s["q"], s["k_cache"], s["tables"],
                                                           s["longest"])
        return pa.prefill_mass(s["mass"], s["q"], s["k_cache"], s["tables"], s["lens"],
                               s["start"], s["longest"], s["scale"], decay=c["decay"],
                               workspace=s["workspace"])
    if "workspace" not in s:
        s["workspace"] = pa.evict_workspace_for(s["k_cache"], s["tables"])
    pa.evict(s["k_cache"], s["v_cache"], s["mass"], s["tables"], s["lens"], s["new_lens"],
             keep_first=c["first"], keep_last=c["last"], workspace=s["workspace"])
    return s["k_cache"], s["v_cache"], s["mass"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _rows_of(pool, table, n, h):
    """The first n tokens of one sequence and head, in 64 bits."""
    blocks = table[:_blocks(n)].long()
    return pool[blocks, h].reshape(-1, pool.shape[-1])[:n].double()


def _exact_bounds(s, c):
    out = s["bounds"].double()
    lens = s["lens"].tolist()
    starts = s["starts"].tolist() if s["starts"] is not None else [0] * len(lens)
    for i, n in enumerate(lens):
        table = s["tables"][i].long()
        lo, full, used = starts[i] // BLOCK, n // BLOCK, _blocks(n)
        if full > lo:
            k = s["k_cache"][table[lo:full]].double()
            out[table[lo:full], :, 0], out[table[lo:full], :, 1] = k.amin(2), k.amax(2)
        if used > full and used > lo:
            k = s["k_cache"][table[full], :, :n - BLOCK * full].double()
            out[table[full], :, 0], out[table[full], :, 1] = k.amin(1), k.amax(1)
    return out


def _exact_select(s, c):
    keep, hkv, d = c["keep"], c["hkv"], c["d"]
    tiles, held = torch.full_like(s["tiles"], -1), torch.zeros_like(s["tile_lens"])
    g = c["hq"] // hkv
    for i, n in enumerate(s["lens"].tolist()):
        used = _blocks(n)
        table = s["tables"][i, :used].long()
        for h in range(hkv):
            if used <= keep:
                chosen = list(range(used))
            else:
                fixed = list(range(c["first"])) + list(range(used - c["last"], used))
                free = torch.arange(c["first"], used - c["last"], device=table.device)
                b = s["bounds"][table[free], h].double()
                q = s["q"][i, h * g:(h + 1) * g].double()
                best = None
                for row in q:
                    x = torch.maximum(row * b[:, 0], row * b[:, 1]).sum(-1)
                    best = x if best is None else torch.maximum(best, x)
                x = best.tolist()
                order = sorted(range(len(x)), key=lambda j: (-x[j], j))[:keep - len(fixed)]
                chosen = sorted(fixed + [j + c["first"] for j in order])
            if chosen:
                at = torch.tensor(chosen, device=table.device)
                tiles[i, h, :len(chosen)] = (table[at] * hkv + h).int()
            held[i, h] = n - BLOCK * (used - len(chosen))
    return tiles, held


def _exact_sparse(s, c):
    out = torch.zeros(s["out"].shape, device=s["out"].device, dtype=torch.float64)
    hkv, d, g = c["hkv"], c["d"], c["hq"] // c["hkv"]
    k, v = (x.reshape(-1, BLOCK, d) for x in (s["k_cache"], s["v_cache"]))
    held = s["tile_lens"].tolist()
    for i in range(c["seqs"]):
        for h in range(hkv):
            n = held[i][h]
            if n == 0:
                continue
            at = s["tiles"][i, h, :_blocks(n)].long()
            kk, vv = (x[at].reshape(-1, d)[:n].double() for x in (k, v))
            q = s["q"][i, h * g:(h + 1) * g].double()
            out[i, h * g:(h + 1) * g] = torch.softmax(q @ kk.T * s["scale"], -1) @ vv
    return out


def _exact_decode(s, c):
    out = torch.zeros(s["out"].shape, device=s["out"].device, dtype=torch.float64)
    mass = s["mass"].double()
    hkv, g = c["hkv"], c["hq"] // c["hkv"]
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        for h in range(hkv):
            k, v = (_rows_of(s[x], s["tables"][i], n, h) for x in ("k_cache", "v_cache"))
            p = torch.softmax(s["q"][i, h * g:(h + 1) * g].double() @ k.T * s["scale"], -1)
            out[i, h * g:(h + 1) * g] = p @ v
            before = mass[i, h, :n].clone() * c["decay"]
            before[n - 1] = 0
            mass[i, h, :n] = before + p.sum(0)
    return out, mass


def _exact_prefill(s, c):
    mass = s["mass"].double()
    hkv, g = c["hkv"], c["hq"] // c["hkv"]
    start = s["start"].tolist()
    for i, n in enumerate(s["lens"].tolist()):
        rows = start[i + 1] - start[i]
        hidden = (torch.arange(n, device=mass.device)[None]
                  > torch.arange(n - rows, n, device=mass.device)[:, None])
        for h in range(hkv):
            k = _rows_of(s["k_cache"], s["tables"][i], n, h)
            new = torch.zeros(n, device=mass.device, dtype=torch.float64)
            for j in range(h * g, h * g + g):
                x = s["q"][start[i]:start[i + 1], j].double() @ k.T * s["scale"]
                new += torch.softmax(x.masked_fill(hidden, -math.inf), -1).sum(0)
            before = mass[i, h, :n].clone() * c["decay"]
            before[n - rows:] = 0
            mass[i, h, :n] = before + new
    return mass


def _exact_evict(s, c):
    lens, new_lens = s["lens"].tolist(), s["new_lens"].tolist()
    k, v, mass = (s[x].clone() for x in ("k_cache", "v_cache", "mass"))
    for i, (n, b) in enumerate(zip(lens, new_lens)):
        if b >= n:
            continue
        last = min(c["last"], b)
        first = min(c["first"], b - last)
        heavy = b - last - first
        table = s["tables"][i].long()
        for h in range(c["hkv"]):
            w = s["mass"][i, h, first:n - last]
            chosen = torch.sort(w, descending=True, stable=True).indices[:heavy] + first
            stays = torch.zeros(n, dtype=torch.bool, device=w.device)
            stays[chosen] = True
            edge = first + heavy
            holes = (~stays[first:edge]).nonzero().flatten() + first
            movers = stays[edge:].nonzero().flatten() + edge
            src = torch.cat([movers, torch.arange(n - last, n, device=w.device)])
            dst = torch.cat([holes, torch.arange(b - last, b, device=w.device)])
            mass[i, h, dst] = s["mass"][i, h, src]
            for new, old in ((k, s["k_cache"]), (v, s["v_cache"])):
                new[table[dst // BLOCK], h, dst % BLOCK] = old[table[src // BLOCK], h, src % BLOCK]
    return k.double(), v.double(), mass.double()


EXACT = {"block_bounds": _exact_bounds, "select_blocks": _exact_select,
         "sparse_decode": _exact_sparse, "decode_mass": _exact_decode,
         "prefill_mass": _exact_prefill, "evict": _exact_evict}


def exact(c, seed):
    return EXACT[c["op"]](prepare(c, seed), c)
