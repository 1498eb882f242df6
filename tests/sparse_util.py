"""Block selection, weight accounting and eviction in 64 bits on the CPU, and how
far a kernel's result may be from them.

Bounds, selections and evictions are exact.  The tolerances of the others are
derived from what the kernels round:
  * a score is an fp32 sum of exact products over head_dim channels, at most 10
    tensor-core steps that each lose up to 2^-22 of the running magnitude, at most
    S = scale * max_t sum |q k|; scaling to base 2, the maximum's way through natural
    units and back and the subtraction of a maximum or of a logarithm (at most S + 17,
    17 for the logarithm of a sum of at most 2^17 weights) lose less than 4 * 2^-22 of
    S + 17: 14 * 2^-22 * (S + 17) in all;
  * the exponential and the reciprocal or logarithm of the sum are good to 2^-21, and P
    enters the product with V rounded to the type (eps / 2); numerator and denominator
    both carry the weights' errors;
  * sums take a rounding (2^-22) for each 16 keys and each rescale or merge, at most
    2 n / 16 + 16 of them.
So a weight is off by `rel` of itself, an output by (rel + eps / 2) of its weights' mean
of |v| and then rounded once; a mass adds one fp32 rounding (2^-24) for each addend.
"""
import math

import torch

BLOCK = 16


def pool(g, nb, hkv, d, dt, poison=()):
    """A pool of random rows; slots listed in poison (block, offset) hold NaN."""
    x = torch.randn(nb, hkv, BLOCK, d, generator=g).to(dt)
    for b, o in poison:
        x[b, :, o] = math.nan
    return x


def tables_for(g, lens, mb=None, spare=3, fill=-1):
    """Block tables with a random pool block for each 16 tokens: (tables, pool size)."""
    used = [(n + BLOCK - 1) // BLOCK for n in lens]
    mb = mb or max(1, max(used))
    nb = sum(used) + spare
    order = torch.randperm(nb, generator=g)
    t, at = torch.full((len(lens), mb), fill, dtype=torch.int32), 0
    for i, n in enumerate(used):
        t[i, :n] = order[at:at + n].int()
        at += n
    return t, nb


def dead_slots(tables, lens, nb):
    """(block, offset) of every slot that no live token is in."""
    live = torch.zeros(nb, BLOCK, dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range((n + BLOCK - 1) // BLOCK):
            live[int(tables[i, j]), :min(BLOCK, n - BLOCK * j)] = True
    return [(int(b), int(o)) for b, o in (~live).nonzero()]


def rows_of(x, table, n, h):
    blocks = table[:(n + BLOCK - 1) // BLOCK].long()
    return x[blocks, h].reshape(-1, x.shape[-1])[:n].double()


def bounds(old, k, tables, lens, starts=None):
    out = old.clone()
    for i, n in enumerate(lens):
        first = 0 if starts is None else min(max(int(starts[i]), 0), n)
        if first >= n:
            continue
        for j in range(first // BLOCK, (n + BLOCK - 1) // BLOCK):
            b = int(tables[i, j])
            live = k[b, :, :min(BLOCK, n - BLOCK * j)].float()
            out[b, :, 0], out[b, :, 1] = (x.to(k.dtype) for x in (live.amin(1), live.amax(1)))
    return out


def select(q, bnd, tables, lens, keep, first, last):
    n, hq, d = q.shape
    hkv = bnd.shape[1]
    g = hq // hkv
    tiles = torch.full((n, hkv, keep), -1, dtype=torch.int32)
    held = torch.zeros(n, hkv, dtype=torch.int32)
    for i, length in enumerate(lens):
        used = (length + BLOCK - 1) // BLOCK
        table = tables[i, :used].long()
        for h in range(hkv):
            chosen = list(range(used))
            if used > keep:
                free = list(range(first, used - last))
                b = bnd[table[free], h].double()
                x = torch.stack([torch.maximum(row * b[:, 0], row * b[:, 1]).sum(-1)
                                 for row in q[i, h * g:(h + 1) * g].double()]).amax(0)
                # what has an infinity or a NaN in it ranks first
                odd = ~(torch.isfinite(b).all(-1).all(-1) &
                        torch.isfinite(q[i, h * g:(h + 1) * g].double()).all())
                x = x.masked_fill(odd, math.inf).tolist()
                order = sorted(range(len(x)), key=lambda j: (-x[j], j))[:keep - first - last]
                chosen = sorted(list(range(first)) + [j + first for j in order] +
                                list(range(used - last, used)))
            at = torch.tensor(chosen, dtype=torch.long)
            tiles[i, h, :len(chosen)] = (table[at] * hkv + h).int()
            held[i, h] = length - BLOCK * (used - len(chosen))
    return tiles, held


def _weights(q, k, scale, hidden=None):
    """Softmax weights of rows q over keys k, and each row's `rel`."""
    x = q @ k.T * scale
    size = q.abs() @ k.abs().T * abs(scale)
    if hidden is not None:
        x, size = x.masked_fill(hidden, -math.inf), size.masked_fill(hidden, 0)
    big, n = size.amax(-1, keepdim=True), k.shape[0]
    rel = 2 * (14 * 2.0 ** -22 * (big + 17) + 2.0 ** -21) + (2 * n / 16 + 16) * 2.0 ** -22
    return torch.softmax(x, -1), rel


def sparse_decode(q, k, v, tiles, held, scale):
    """(result, tolerance before the last rounding), in 64 bits."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    out, tol = (torch.zeros(n, hq, d, dtype=torch.float64) for _ in range(2))
    kk, vv = (x.reshape(-1, BLOCK, d) for x in (k, v))
    for i in range(n):
        for h in range(hkv):
            m = int(held[i, h])
            if m == 0:
                continue
            at = tiles[i, h, :(m + BLOCK - 1) // BLOCK].long()
            a, b = (x[at].reshape(-1, d)[:m].double() for x in (kk, vv))
            p, rel = _weights(q[i, h * g:(h + 1) * g].double(), a, scale)
            out[i, h * g:(h + 1) * g] = p @ b
            tol[i, h * g:(h + 1) * g] = (rel + torch.finfo(q.dtype).eps / 2) * (p @ b.abs())
    return out, tol


def _account(mass, tol, i, h, n, new, err, addends, decay, fresh):
    before = torch.zeros(n, dtype=torch.float64)
    if decay != 0.0:
        before = mass[i, h, :n].clone() * decay
    before[n - fresh:] = 0
    mass[i, h, :n] = before + new
    tol[i, h, :n] = err + (addends + 2) * 2.0 ** -24 * (new + before.abs())


def decode_mass(q, mass, k, v, tables, lens, scale, decay):
    """(out, its tolerance, mass, its tolerance)."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    out, tol = (torch.zeros(n, hq, d, dtype=torch.float64) for _ in range(2))
    mass = mass.double().clone()
    mtol = torch.zeros_like(mass)
    for i, m in enumerate(lens):
        for h in range(hkv if m else 0):
            a, b = (rows_of(x, tables[i], m, h) for x in (k, v))
            p, rel = _weights(q[i, h * g:(h + 1) * g].double(), a, scale)
            out[i, h * g:(h + 1) * g] = p @ b
            tol[i, h * g:(h + 1) * g] = (rel + torch.finfo(q.dtype).eps / 2) * (p @ b.abs())
            _account(mass, mtol, i, h, m, p.sum(0), (p * rel).sum(0), g, decay, 1)
    return out, tol, mass, mtol


def prefill_mass(q, mass, k, tables, lens, start, scale, decay):
    hq, hkv = q.shape[1], k.shape[1]
    g = hq // hkv
    mass = mass.double().clone()
    mtol = torch.zeros_like(mass)
    for i, m in enumerate(lens):
        rows = start[i + 1] - start[i]
        if rows == 0:
            continue
        hidden = torch.arange(m)[None] > torch.arange(m - rows, m)[:, None]
        for h in range(hkv):
            a = rows_of(k, tables[i], m, h)
            new, err = (torch.zeros(m, dtype=torch.float64) for _ in range(2))
            for j in range(h * g, h * g + g):
                p, rel = _weights(q[start[i]:start[i + 1], j].double(), a, scale, hidden)
                new += p.sum(0)
                err += (p * rel).sum(0)
            _account(mass, mtol, i, h, m, new, err, rows * g, decay, rows)
    return mass, mtol


def evict(k, v, mass, tables, lens, new_lens, keep_first, keep_last):
    k, v, mass = k.clone(), v.clone(), mass.clone()
    for i, (n, b) in enumerate(zip(lens, new_lens)):
        if b >= n:
            continue
        last = min(keep_last, b)
        first = min(keep_first, b - last)
        edge = b - last
        table = tables[i].long()
        for h in range(mass.shape[1]):
            w = mass[i, h].clone()
            x = [math.inf if math.isnan(y) else y for y in w[first:n - last].tolist()]
            odd = [math.isnan(y) for y in w[first:n - last].tolist()]
            order = sorted(range(len(x)), key=lambda j: (not odd[j], -x[j], j))
            stays = {j + first for j in order[:edge - first]}
            holes = [t for t in range(first, edge) if t not in stays]
            movers = sorted(t for t in stays if t >= edge)
            assert len(holes) == len(movers)
            src = torch.tensor(movers + list(range(n - last, n)), dtype=torch.long)
            dst = torch.tensor(holes + list(range(b - last, b)), dtype=torch.long)
            mass[i, h, dst] = w[src]
            for pool_ in (k, v):
                rows = pool_[table[src // BLOCK], h, src % BLOCK].clone()
                pool_[table[dst // BLOCK], h, dst % BLOCK] = rows
    return k, v, mass


def close(got, ref, tol, what=""):
    """A rounded result against its reference and the tolerance before that rounding."""
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    t = torch.finfo(got.dtype).eps / 2 * (ref.abs() + tol) + 1.02 * tol + 2.0 ** -25
    d = (got.double().cpu() - ref).abs()
    assert bool((d <= t).all()), f"{what}: off by {float((d / t).max())} of the tolerance"


def mass_close(got, ref, tol, what=""):
    got = got.double().cpu()
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    d = (got - ref).abs()
    ok = same | (d <= 1.02 * tol + 2.0 ** -126)
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} beyond the tolerance"


def bits(x):
    """Raw contents, NaN payloads too."""
    return x.contiguous().view(torch.int32 if x.dtype == torch.float32 else torch.int16).cpu()
