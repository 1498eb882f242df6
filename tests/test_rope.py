"""pa_rope_and_cache and pa_qk_norm_rope refuse what they cannot do, on the
host, before anything is launched (no GPU needed)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_260_gb300 import _build
    import paged_kv_cache_260_gb300 as pa
    _build.build()
    return pa.load()


FAKE = 0x1000


def _append(lib, **kw):
    a = dict(q_out=FAKE, q=FAKE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, pos=FAKE, cs=FAKE,
             qn=None, kn=None, tokens=4, hq=8, hkv=2, d=128, maps=1, bs=16, nb=64, table=32,
             rot=128, inter=0, eps=1e-6, qs=1024, ks=256, vs=256, qos=1024, dtype=0)
    a.update(kw)
    v = list(a.values())
    return lib.pa_rope_and_cache(*v[:11], *v[11:21], C.c_float(v[21]), *v[22:26], v[26], None)


def _rope(lib, **kw):
    a = dict(q_out=FAKE, k_out=FAKE, q=FAKE, k=FAKE, pos=FAKE, cs=FAKE, qn=None, kn=None, tokens=4,
             hq=8, hkv=2, d=128, maps=1, table=32, rot=128, inter=0, eps=1e-6, qs=1024, ks=256,
             qos=1024, kos=256, dtype=0)
    a.update(kw)
    v = list(a.values())
    return lib.pa_qk_norm_rope(*v[:8], *v[8:16], C.c_float(v[16]), *v[17:21], v[21], None)


@pytest.mark.parametrize("call", [_append, _rope])
@pytest.mark.parametrize("kw,status", [
    (dict(d=96, rot=64), 2), (dict(dtype=5), 2), (dict(maps=3), 2), (dict(maps=0), 2),
    (dict(rot=24), 2),                                     # rotary_dim not a multiple of 16
    (dict(rot=0), 1), (dict(rot=-16), 1), (dict(rot=144), 1), (dict(rot=128, maps=2), 1),
    (dict(hkv=0), 1), (dict(hq=0), 1), (dict(hq=7), 1), (dict(tokens=-1), 1), (dict(table=0), 1),
    (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(pos=None), 1), (dict(cs=None), 1),
    (dict(q_out=None), 1), (dict(q=0x1008), 1), (dict(qn=0x1002), 1), (dict(kn=0x1002), 1),
    (dict(cs=0x1004), 1), (dict(pos=0x1002), 1),
    (dict(qs=1023), 1), (dict(qs=1028), 1), (dict(ks=255), 1), (dict(qos=1016), 1), (dict(qs=0), 1),
    (dict(qs=2048), 1),                                    # q_out is q, with another stride
    (dict(tokens=0, q=None, k=None), 0)])
def test_both_refuse(lib, call, kw, status):
    assert call(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(bs=32), 2), (dict(nb=0), 1), (dict(v=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(slots=None), 1), (dict(slots=0x1004), 1), (dict(vs=248), 1), (dict(vc=0x1004), 1)])
def test_append_refuses(lib, kw, status):
    assert _append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(k_out=None), 1), (dict(kos=128), 1),
                                       (dict(ks=512), 1), (dict(k_out=0x1008), 1)])
def test_rope_refuses(lib, kw, status):
    assert _rope(lib, **kw) == status


def test_bindings_refuse_host_tensors():
    import paged_kv_cache_260_gb300 as pa
    q = torch.zeros(2, 8, 64, dtype=torch.float16)
    k = torch.zeros(2, 2, 64, dtype=torch.float16)
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    pos = torch.zeros(2, dtype=torch.int32)
    cs = torch.zeros(8, 64)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(q, k, q, k, pos, cs)
    with pytest.raises(ValueError):
        pa.rope_and_cache(q, q, k, k, pool, pool, pos.long(), pos, cs)


def _packed(entry, size=None, **kw):
    from paged_kv_cache_260_gb300 import _ROPE_ARGS
    a = dict(q_out=FAKE, k_out=FAKE, q=FAKE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, pos=FAKE,
             cs=FAKE, qn=0, kn=0, stream=0, qs=1024, ks=256, vs=256, qos=1024, kos=256, eps=1e-6,
             tokens=0, hq=8, hkv=2, d=128, maps=1, bs=16, nb=64, table=32, rot=128, inter=0,
             dtype=0)
    a.update(kw)
    return entry(_ROPE_ARGS.pack(_ROPE_ARGS.size if size is None else size, *a.values()))


@pytest.mark.parametrize("name", ["pa_rope_and_cache_args", "pa_qk_norm_rope_args"])
@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(size=0), 1), (dict(size=200), 1), (dict(tokens=-1), 1), (dict(hq=7), 1),
    (dict(hkv=0), 1), (dict(d=96, rot=64), 2), (dict(maps=3), 2), (dict(rot=24), 2),
    (dict(table=0), 1), (dict(dtype=5), 2), (dict(eps=-1.0), 1), (dict(eps=1e300), 1),
    (dict(tokens=4, q=0), 1), (dict(tokens=4, k=0x1008), 1), (dict(tokens=4, q_out=0), 1),
    (dict(tokens=4, pos=0), 1), (dict(tokens=4, cs=0x1004), 1), (dict(tokens=4, qn=0x1002), 1),
    (dict(tokens=4, kn=0x1002), 1), (dict(tokens=4, qs=1028), 1), (dict(tokens=4, ks=255), 1),
    (dict(tokens=4, qos=1016), 1)])
def test_packed_arguments_arrive(lib, name, kw, status):
    assert _packed(getattr(lib, name), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(bs=32), 2), (dict(nb=0), 1), (dict(tokens=4, v=0), 1), (dict(tokens=4, kc=0x1004), 1),
    (dict(tokens=4, vc=0), 1), (dict(tokens=4, slots=0), 1), (dict(tokens=4, vs=248), 1)])
def test_packed_arguments_of_the_pool_arrive(lib, kw, status):
    assert _packed(lib.pa_rope_and_cache_args, **kw) == status


def test_packed_arguments_null(lib):
    assert lib.pa_rope_and_cache_args(None) == 1
    assert lib.pa_qk_norm_rope_args(None) == 1
    assert _packed(lib.pa_qk_norm_rope_args, tokens=4, k_out=0) == 1
    assert _packed(lib.pa_qk_norm_rope_args, tokens=4, kos=248) == 1
