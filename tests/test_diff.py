"""The differential entry points refuse what they cannot do, on the host, and
their reference is what the formula says (no GPU needed)."""
import ctypes as C
import math

import pytest
import torch

from diff_util import reference

FAKE = 0x1000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_260_gb300 import _build
    import paged_kv_cache_260_gb300 as pa
    _build.build()
    return pa.load()


def _decode(lib, **kw):
    a = dict(out=0x2000, q=FAKE, k=FAKE, v=FAKE, tables=FAKE, lens=FAKE, lam=FAKE, w=None, n=4, hq=8,
             hkv=2, d=128, bs=16, mb=8, nb=64, scale=0.1, eps=1e-6, os=1.0, dtype=0, ws=None,
             wb=0)
    a.update(kw)
    v = list(a.values())
    return lib.pa_diff_decode(*v[:15], *(C.c_float(x) for x in v[15:18]), *v[18:], None)


def _prefill(lib, **kw):
    a = dict(out=0x2000, q=FAKE, k=FAKE, v=FAKE, tables=FAKE, lens=FAKE, start=FAKE, lam=FAKE, w=None,
             n=4, longest=32, hq=8, hkv=2, d=128, bs=16, mb=8, nb=64, scale=0.1, eps=1e-6, os=1.0,
             dtype=0, ws=None, wb=0)
    a.update(kw)
    v = list(a.values())
    return lib.pa_diff_prefill(*v[:17], *(C.c_float(x) for x in v[17:20]), *v[20:], None)


@pytest.mark.parametrize("call", [_decode, _prefill])
@pytest.mark.parametrize("kw,status", [
    (dict(d=96), 2), (dict(bs=8), 2), (dict(dtype=3), 2), (dict(hq=7), 1), (dict(n=-1), 1),
    (dict(mb=0), 1), (dict(nb=0), 1), (dict(hkv=0), 1), (dict(scale=math.nan), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.inf), 1), (dict(os=math.nan), 1), (dict(lam=None), 1),
    (dict(lam=0x1002), 1), (dict(w=0x1008), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(out=FAKE), 1),
    (dict(q=0x1008), 1), (dict(tables=None), 1), (dict(lens=0x1001), 1),
    (dict(n=0, lam=None), 0), (dict(n=0, d=96), 2)])
def test_both_refuse(lib, call, kw, status):
    assert call(lib, **kw) == status


def test_decode_refuses_wide_groups(lib):
    assert _decode(lib, hq=34) == 2                          # group 17
    assert _decode(lib, hq=32, q=None) == 1                  # group 16 is served
    assert lib.pa_diff_decode_workspace_size(0, 8, 2, 128, 8) == 0
    assert lib.pa_diff_decode_workspace_size(4, 7, 2, 128, 8) == 0
    assert lib.pa_diff_decode_workspace_size(4, 2 ** 31 - 2, 2, 128, 8) == 0


def test_prefill_refuses(lib):
    assert _prefill(lib, start=None) == 1
    assert _prefill(lib, scale=0.0) == 1 and _prefill(lib, scale=-1.0) == 1
    assert _prefill(lib, hq=258, hkv=1) == 2
    assert _prefill(lib, longest=-1) == 1 and _prefill(lib, longest=0) == 0
    assert _prefill(lib, ws=0x1010, wb=4096) == 3            # misaligned workspace
    assert _prefill(lib, ws=0x1000, wb=16) == 3
    # 16 + 4 * seqs * query tile pairs + 8 * seqs, rounded up to 256
    assert lib.pa_diff_prefill_workspace_size(8, 512, 32, 8) == 512     # 16 + 256 + 64
    assert lib.pa_diff_prefill_workspace_size(8, 512, 30, 8) == 0


def test_bindings_refuse_host_tensors():
    import paged_kv_cache_260_gb300 as pa
    q = torch.zeros(2, 8, 64, dtype=torch.float16)
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    t = torch.zeros(2, 2, dtype=torch.int32)
    lens = torch.ones(2, dtype=torch.int32)
    lam = torch.zeros(8)
    with pytest.raises(ValueError):
        pa.diff_decode(q, q, pool, pool, t, lens, lam, 1.0)
    with pytest.raises(ValueError):
        pa.diff_prefill(q, q, pool, pool, t, lens, torch.arange(3).int(), 1, lam, 1.0,
                        workspace=None)


def test_reference_by_hand():
    # one head, three tokens, two channels a map; everything written out
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, 1, 4, generator=g)
    k = torch.randn(2, 1, 16, 4, generator=g)
    v = torch.randn(2, 1, 16, 4, generator=g)
    tables = torch.tensor([[1, 0]])
    ref, tol = reference(q, k, v, tables, 0, [2], torch.tensor([0.7]), 0.5, None, 0.0, 2.0, 0.0)
    want = [0.0] * 4
    for lo, f in ((0, 1.0), (2, -0.7)):
        s = [0.5 * sum(float(q[0, 0, lo + c]) * float(k[1, 0, t, lo + c]) for c in range(2))
             for t in range(3)]
        z = sum(math.exp(x) for x in s)
        for c in range(4):
            want[c] += 2.0 * f * sum(math.exp(s[t]) / z * float(v[1, 0, t, c]) for t in range(3))
    assert all(abs(float(ref[0, 0, c]) - want[c]) < 1e-6 for c in range(4))
    w = torch.tensor([1.0, 2.0, 0.5, -1.0])
    ref, _ = reference(q, k, v, tables, 0, [2], torch.tensor([0.7]), 0.5, w, 0.1, 2.0, 0.0)
    r = math.sqrt(sum((x / 2) ** 2 for x in want) / 4 + 0.1)
    assert all(abs(float(ref[0, 0, c]) - want[c] / r * float(w[c])) < 1e-6 for c in range(4))
    # equal maps and lambda 1 leave nothing
    q[..., 2:], k[..., 2:] = q[..., :2], k[..., :2]
    ref, _ = reference(q, k, v, tables, 0, [2], torch.tensor([1.0]), 0.5, None, 0.0, 1.0, 0.0)
    assert float(ref.abs().max()) < 1e-12


def _packed(entry, size=None, **kw):
    from paged_kv_cache_260_gb300 import _DIFF_ARGS
    a = dict(out=0x2000, q=FAKE, k=FAKE, v=FAKE, tables=FAKE, lens=FAKE, start=FAKE, lam=FAKE, w=0,
             ws=0, stream=0, wb=0, scale=0.1, eps=1e-6, os=1.0, n=4, longest=32, hq=8, hkv=2, d=128,
             bs=16, mb=8, nb=64, dtype=0)
    a.update(kw)
    return entry(_DIFF_ARGS.pack(_DIFF_ARGS.size if size is None else size, *a.values()))


@pytest.mark.parametrize("name", ["pa_diff_decode_args", "pa_diff_prefill_args"])
@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 0), (dict(n=0, size=0), 1), (dict(n=0, size=184), 1), (dict(n=-1), 1),
    (dict(hq=7), 1), (dict(hkv=0), 1), (dict(d=96), 2), (dict(bs=8), 2), (dict(mb=0), 1),
    (dict(nb=0), 1), (dict(dtype=3), 2), (dict(scale=math.nan), 1), (dict(eps=-1.0), 1),
    (dict(os=1e300), 1), (dict(out=0), 1), (dict(out=FAKE), 1), (dict(q=0x1008), 1),
    (dict(k=0), 1), (dict(v=0x1008), 1), (dict(tables=0), 1), (dict(lens=0x1001), 1),
    (dict(lam=0), 1), (dict(w=0x1008), 1)])
def test_packed_arguments_arrive(lib, name, kw, status):
    assert _packed(getattr(lib, name), **kw) == status


def test_packed_arguments_of_one(lib):
    assert lib.pa_diff_decode_args(None) == 1 and lib.pa_diff_prefill_args(None) == 1
    assert _packed(lib.pa_diff_decode_args, hq=34) == 2
    assert _packed(lib.pa_diff_prefill_args, start=0) == 1
    assert _packed(lib.pa_diff_prefill_args, longest=-1) == 1
    assert _packed(lib.pa_diff_prefill_args, longest=0) == 0
    assert _packed(lib.pa_diff_prefill_args, ws=0x1010, wb=4096) == 3
    assert _packed(lib.pa_diff_prefill_args, ws=0x1000, wb=16) == 3
