"""Differential attention in 64 bits, and how far a kernel's result may be
from it.

The tolerance is derived, element by element, from what the kernels round:
  * a score is an fp32 sum of exact products over head_dim / 2 channels, at most
    10 tensor-core steps that each lose up to 2^-22 of the running magnitude,
    which is at most S = scale * max_t sum |q k|; the scaling to base 2 and the
    subtraction of the maximum lose less than 2^-22 S again: 12 * 2^-22 * S;
  * the exponential is good to 2^-21 and what rounds P before the product with
    V to `p_round`; numerator and denominator both carry the weights' errors;
  * the accumulators take a rounding (2^-22) for each 16-key step and each
    rescale or merge, at most 2 n / 16 + 16 of them.
So each map's result is off by at most `rel` times its weights' mean of |v|;
with a norm the row's factor carries the same errors, averaged; the result is
rounded once, by at most eps / 2 of its value (half the smallest fp16 subnormal,
2^-25, below the normal range).
"""
import math

import torch


def reference(q, k_cache, v_cache, tables, seq, pos, lam, scale, w, eps, out_scale, p_round):
    """Rows q [rows, hq, d] of sequence `seq` at positions pos: (result, tolerance before the
    last rounding), both [rows, hq, d] in 64 bits."""
    rows, hq, d = q.shape
    hkv = k_cache.shape[1]
    g, half = hq // hkv, d // 2
    ref, tol = (torch.zeros(rows, hq, d, dtype=torch.float64) for _ in range(2))
    n = int(max(pos)) + 1 if rows else 0
    if n <= 0:
        return ref, tol
    blocks = tables[seq, :(n + 15) // 16].long()
    assert bool((blocks >= 0).all())
    hidden = torch.arange(n)[None] > torch.as_tensor(pos)[:, None]
    for h in range(hkv):
        k = k_cache[blocks, h].reshape(-1, d)[:n].double()
        v = v_cache[blocks, h].reshape(-1, d)[:n].double()
        for j in range(h * g, h * g + g):
            y, e = (torch.zeros(rows, d, dtype=torch.float64) for _ in range(2))
            for part, f in ((slice(0, half), 1.0), (slice(half, d), -float(lam[j]))):
                a, b = q[:, j, part].double(), k[:, part]
                s = (a @ b.T * scale).masked_fill(hidden, -math.inf)
                big = (a.abs() @ b.abs().T * abs(scale)).masked_fill(hidden, 0).amax(-1, True)
                p = torch.softmax(s, -1)
                rel = 2 * (12 * 2.0 ** -22 * big + 2.0 ** -21) + p_round + \
                    (2 * n / 16 + 16) * 2.0 ** -22
                y += f * (p @ v)
                e += abs(f) * rel * (p @ v.abs())
            if w is not None:
                r = torch.sqrt((y ** 2).mean(-1, keepdim=True) + eps)
                ww = w.double()
                # d(y/r) = dy/r - y (mean y dy) / r^3, and the norm's own roundings
                e = ww.abs() * (e / r + y.abs() * ((y.abs() * e).mean(-1, True) / r ** 3) +
                                2.0 ** -19 * y.abs() / r)
                y = y / r * ww
            ref[:, j] = y * out_scale
            tol[:, j] = e * abs(out_scale) + 2.0 ** -20 * ref[:, j].abs()
    return ref, tol


def assert_close(got, ref, tol, what=""):
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite output"
    # second-order terms of the bound: one part in 50
    t = torch.finfo(got.dtype).eps / 2 * (ref.abs() + tol) + 1.02 * tol + 2.0 ** -25
    d = (got.double().cpu() - ref).abs()
    assert bool((d <= t).all()), f"{what}: off by {float((d / t).max())} of the tolerance"
