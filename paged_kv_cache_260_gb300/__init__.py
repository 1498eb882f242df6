"""GB300 (sm_103a) paged KV cache: decode attention, chunked prefill, both
also as differential attention, reshape_and_cache, rope_and_cache,
copy_blocks, swap_blocks.

A thin ctypes binding over ``libpagedattn.so`` (the C ABI in
``include/pagedattn.h``).  Functions take torch CUDA tensors, pass their data
pointers, sizes and the current stream to the library and raise
``PagedAttnError`` on a non-zero status.  No computation happens here: every
step runs in the library's kernels, and there is no fallback when the library
is missing -- loading it fails loudly.

Names follow the C ABI without the ``pa_`` prefix.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading

__all__ = [
    "PagedAttnError", "load", "version", "decode", "decode_workspace_size", "workspace_for",
    "decode_noalloc", "decode_append", "decode_shared_prefix",
    "decode_shared_prefix_workspace_size", "diff_decode", "diff_decode_workspace_size",
    "diff_decode_workspace_for", "prefill", "prefill_workspace_size", "diff_prefill",
    "diff_prefill_workspace_size", "diff_prefill_workspace_for",
    "reshape_and_cache", "rope_and_cache", "qk_norm_rope", "copy_blocks", "swap_blocks",
    "gather_kv", "validate_tables", "selftest_bounded_wait", "get_device_error",
    "PA_DTYPE_F16", "PA_DTYPE_BF16", "DEVERR", "STATUS",
]

PA_DTYPE_F16 = 0
PA_DTYPE_BF16 = 1
BLOCK_SIZE = 16
STATUS = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_WORKSPACE",
          4: "PA_ERR_CUDA", 5: "PA_ERR_DEVICE"}
DEVERR = {"SLOT_RANGE": 0x1, "BLOCK_RANGE": 0x2, "TABLE_RANGE": 0x4, "SEQLEN_RANGE": 0x8,
          "TIMEOUT": 0x10, "APPEND_SLOT": 0x20, "QUERY_RANGE": 0x40,
          "POSITION_RANGE": 0x80}

# struct pa_rope_args and struct pa_diff_args: one packed argument costs a call 2 us
# less than ctypes' conversion of 27
_ROPE_ARGS = struct.Struct("Q13P5qd11i0Q")
_DIFF_ARGS = struct.Struct("Q11PQ3d9i0Q")

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedattn.so")
_lib = None
_lock = threading.Lock()


class PagedAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        name = STATUS.get(status, str(status))
        super().__init__(f"{fn} failed: {name}")


def load(path: str = LIB_PATH):
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    L = _lib
    if L is not None:                    # every call after the first
        return L
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(path)
        vp, i, f, sz = C.c_void_p, C.c_int, C.c_float, C.c_size_t
        L.pa_version.restype = i
        L.pa_version.argtypes = []
        L.pa_status_string.restype = C.c_char_p
        L.pa_status_string.argtypes = [i]
        L.pa_decode_workspace_size.restype = sz
        L.pa_decode_workspace_size.argtypes = [i, i, i, i, i, i]
        L.pa_decode.restype = i
        L.pa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, vp, sz, vp]
        L.pa_decode_append.restype = i
        L.pa_decode_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                       f, i, i, vp, sz, vp]
        L.pa_decode_shared_prefix_workspace_size.restype = sz
        L.pa_decode_shared_prefix_workspace_size.argtypes = [i, i, i, i, i, i, i]
        L.pa_decode_shared_prefix.restype = i
        L.pa_decode_shared_prefix.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i,
                                              i, i, i, i, f, i, vp, sz, vp]
        L.pa_decode_noalloc.restype = i
        L.pa_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp]
        L.pa_reshape_and_cache.restype = i
        L.pa_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        i64 = C.c_int64
        L.pa_rope_and_cache.restype = i
        L.pa_rope_and_cache.argtypes = [vp] * 11 + [i] * 10 + [f] + [i64] * 4 + [i, vp]
        L.pa_qk_norm_rope.restype = i
        L.pa_qk_norm_rope.argtypes = [vp] * 8 + [i] * 8 + [f] + [i64] * 4 + [i, vp]
        L.pa_diff_decode.restype = i
        L.pa_diff_decode.argtypes = [vp] * 8 + [i] * 7 + [f] * 3 + [i, vp, sz, vp]
        L.pa_diff_prefill.restype = i
        L.pa_diff_prefill.argtypes = [vp] * 9 + [i] * 8 + [f] * 3 + [i, vp, sz, vp]
        for name in ("pa_rope_and_cache_args", "pa_qk_norm_rope_args", "pa_diff_decode_args",
                     "pa_diff_prefill_args"):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = i, [C.c_char_p]
        L.pa_copy_blocks.restype = i
        L.pa_copy_blocks.argtypes = [vp, vp, vp, i, i, i, i, i, i, vp]
        L.pa_swap_blocks.restype = i
        L.pa_swap_blocks.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
        L.pa_gather_kv.restype = i
        L.pa_gather_kv.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
        L.pa_validate_tables.restype = i
        L.pa_validate_tables.argtypes = [vp, vp, i, i, i, i, vp, vp]
        L.pa_prefill.restype = i
        L.pa_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, vp,
                                 sz, vp]
        L.pa_prefill_workspace_size.restype = sz
        L.pa_prefill_workspace_size.argtypes = [i, i, i, i]
        L.pa_diff_decode_workspace_size.restype = sz
        L.pa_diff_decode_workspace_size.argtypes = [i] * 5
        L.pa_diff_prefill_workspace_size.restype = sz
        L.pa_diff_prefill_workspace_size.argtypes = [i] * 4
        L.pa_selftest_bounded_wait.restype = i
        L.pa_selftest_bounded_wait.argtypes = [i, vp]
        L.pa_get_device_error.restype = i
        L.pa_get_device_error.argtypes = [vp, C.POINTER(C.c_uint32), i]
        _lib = L
        return L


def version() -> int:
    return load().pa_version()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return PA_DTYPE_F16
    if t.dtype == torch.bfloat16:
        return PA_DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    # a plain int: the argtypes (c_void_p) convert it
    return None if t is None else t.data_ptr()


_current_raw_stream = None


def _stream(stream):
    """The stream's handle; by default the current device's current stream,
    read as a raw handle (building a torch.cuda.Stream object for it costs a
    few microseconds a call)."""
    global _current_raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and dev is not None:
            torch.cuda.init()
            _current_raw_stream = lambda: raw(dev())
        else:
            _current_raw_stream = lambda: torch.cuda.current_stream().cuda_stream
    return _current_raw_stream()


class _Names:
    """What the hot wrappers look up in torch, once."""

    def __init__(self):
        torch = _torch()
        self.i32, self.i64, self.f32 = torch.int32, torch.int64, torch.float32
        self.codes = {torch.float16: PA_DTYPE_F16, torch.bfloat16: PA_DTYPE_BF16}
        self.device = torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream


_names = None


def _hot():
    global _names
    if _names is None:
        _names = _Names()
    return _names


def _scratch(nbytes, device, stream):
    """A uint8 scratch tensor for one call, out of the call's stream's memory: the
    caching allocator may otherwise hand out memory that kernels on the
    current stream still use, or hand this out again before the call's kernels
    have run."""
    torch = _torch()
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _check(fn: str, rc: int):
    if rc != 0:
        raise PagedAttnError(fn, rc)


def _require(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                          partition_size=0) -> int:
    return int(load().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                               max_blocks_per_seq, partition_size))


def workspace_for(q, k_cache, block_tables, partition_size=0, stream=None):
    """A workspace tensor sized for pa_decode on these shapes (None when none is needed)."""
    n, hq, d = q.shape
    nbytes = decode_workspace_size(n, hq, k_cache.shape[1], d, block_tables.shape[1],
                                   partition_size)
    if nbytes == 0:
        return None
    return _scratch(nbytes, q.device, stream)


def decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale, partition_size=0,
           workspace=None, stream=None):
    """pa_decode: out[s, h] = softmax(scale * q[s, h] . K_s) V_s over the paged pool.

    q, out [num_seqs, num_heads, head_dim]; k_cache, v_cache
    [num_blocks, num_kv_heads, 16, head_dim]; block_tables int32
    [num_seqs, max_blocks]; seq_lens int32 [num_seqs].
    """
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _require(out.shape == q.shape and d2 == d and v_cache.shape == k_cache.shape, "shapes")
    _require(block_tables.dim() == 2 and block_tables.shape[0] == n and seq_lens.shape == (n,),
             "table shapes")
    for t in (out, q, k_cache, v_cache, block_tables, seq_lens):
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")
    if workspace is None:
        workspace = workspace_for(q, k_cache, block_tables, partition_size, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().pa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                          _ptr(seq_lens), n, hq, hkv, d, bs, block_tables.shape[1], nb,
                          float(scale), _dtype_code(q), int(partition_size), _ptr(workspace),
                          wbytes, _stream(stream))
    _check("pa_decode", rc)
    return out


def decode_append(out, q, k_cache, v_cache, block_tables, seq_lens, k_new, v_new, slot_mapping,
                  scale, partition_size=0, workspace=None, stream=None):
    """pa_decode_append: reshape_and_cache of each sequence's newest token, then decode,
    in one launch.  slot_mapping[s] is the slot of position seq_lens[s] - 1 (or < 0)."""
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _require(out.shape == q.shape and d2 == d and v_cache.shape == k_cache.shape, "shapes")
    _require(block_tables.dim() == 2 and block_tables.shape[0] == n and seq_lens.shape == (n,),
             "table shapes")
    _require(k_new.shape == (n, hkv, d) and v_new.shape == k_new.shape and
             slot_mapping.shape == (n,), "new-token shapes")
    if workspace is None:
        workspace = workspace_for(q, k_cache, block_tables, partition_size, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().pa_decode_append(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(block_tables), _ptr(seq_lens), _ptr(k_new), _ptr(v_new),
                                 _ptr(slot_mapping), n, hq, hkv, d, bs, block_tables.shape[1], nb,
                                 float(scale), _dtype_code(q), int(partition_size),
                                 _ptr(workspace), wbytes, _stream(stream))
    _check("pa_decode_append", rc)
    return out


def decode_shared_prefix_workspace_size(num_seqs, group_size, prefix_len, num_heads,
                                        num_kv_heads, head_dim, max_blocks_per_seq) -> int:
    return int(load().pa_decode_shared_prefix_workspace_size(
        num_seqs, group_size, prefix_len, num_heads, num_kv_heads, head_dim, max_blocks_per_seq))


def decode_shared_prefix(out, q, k_cache, v_cache, block_tables, seq_lens, group_size,
                         prefix_len, scale, k_new=None, v_new=None, slot_mapping=None,
                         workspace=None, stream=None):
    """pa_decode_shared_prefix: decode (with the newest tokens appended when
    k_new, v_new and slot_mapping are given) of a batch whose consecutive
    groups of `group_size` sequences share their first `prefix_len` tokens'
    blocks; the shared prefix is read once per group."""
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _require(out.shape == q.shape and d2 == d and v_cache.shape == k_cache.shape, "shapes")
    _require(block_tables.dim() == 2 and block_tables.shape[0] == n and seq_lens.shape == (n,),
             "table shapes")
    if k_new is not None:
        _require(k_new.shape == (n, hkv, d) and v_new.shape == k_new.shape and
                 slot_mapping.shape == (n,), "new-token shapes")
    if workspace is None:
        nbytes = decode_shared_prefix_workspace_size(n, group_size, prefix_len, hq, hkv, d,
                                                     block_tables.shape[1])
        workspace = _scratch(nbytes, q.device, stream) if nbytes else None
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().pa_decode_shared_prefix(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens),
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n, int(group_size), int(prefix_len), hq,
        hkv, d, bs, block_tables.shape[1], nb, float(scale), _dtype_code(q), _ptr(workspace),
        wbytes, _stream(stream))
    _check("pa_decode_shared_prefix", rc)
    return out


def prefill_workspace_size(num_seqs, max_query_len, num_heads, num_kv_heads) -> int:
    return int(load().pa_prefill_workspace_size(num_seqs, max_query_len, num_heads, num_kv_heads))


def prefill(out, q, k_cache, v_cache, block_tables, seq_lens, query_start, max_query_len, scale,
            workspace="auto", stream=None):
    """pa_prefill: causal attention of each sequence's newest chunk over the paged pool.

    q, out [total_q, num_heads, head_dim], the chunks packed back to back;
    query_start int32 [num_seqs + 1]; seq_lens int32 [num_seqs] counts the
    chunk; max_query_len (host int) is the longest chunk.  workspace: "auto"
    allocates the work-order buffer, None runs without it, or a CUDA uint8
    tensor of at least prefill_workspace_size(...) bytes.
    """
    t, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    n = seq_lens.shape[0]
    _require(out.shape == q.shape and d2 == d and v_cache.shape == k_cache.shape, "shapes")
    _require(block_tables.dim() == 2 and block_tables.shape[0] == n and
             query_start.shape == (n + 1,), "table shapes")
    for x in (out, q, k_cache, v_cache, block_tables, seq_lens, query_start):
        _require(x.is_cuda and x.is_contiguous(), "tensors must be contiguous CUDA tensors")
    if isinstance(workspace, str):
        nbytes = prefill_workspace_size(n, int(max_query_len), hq, hkv)
        workspace = _scratch(nbytes, q.device, stream) if nbytes else None
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().pa_prefill(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                           _ptr(seq_lens), _ptr(query_start), n, int(max_query_len), hq, hkv, d,
                           bs, block_tables.shape[1], nb, float(scale), _dtype_code(q),
                           _ptr(workspace), wbytes, _stream(stream))
    _check("pa_prefill", rc)
    return out


_NEAR = "tensors must be contiguous, of the right type and on the current CUDA device"


def _near(t, dtype, device):
    """The address of a contiguous tensor of this type on this device."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(_NEAR)
    return t.data_ptr()


def _current(t, names):
    """The device of t, which has to be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != names.device():
        raise ValueError("tensors must be on the current CUDA device")
    return dev


def _code(dtype, names):
    code = names.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _weights(w, size, dtype, device):
    """The address of norm weights [size]."""
    if w.shape != (size,):
        raise ValueError(f"norm weights: [{size}]")
    return _near(w, dtype, device)


def _diff_pointers(out, q, k_cache, v_cache, block_tables, seq_lens, lam, norm_weight, names):
    """Checks what diff_decode and diff_prefill share; the device and the addresses."""
    i32 = names.i32
    shape, pool, tables = q.shape, k_cache.shape, block_tables.shape
    dt, dev = q.dtype, _current(q, names)
    if (out.shape != shape or pool[3] != shape[2] or v_cache.shape != pool or len(tables) != 2 or
            seq_lens.shape != tables[:1] or lam.shape != shape[1:2]):
        raise ValueError("shapes")
    if (out.dtype is not dt or k_cache.dtype is not dt or v_cache.dtype is not dt or
            block_tables.dtype is not i32 or seq_lens.dtype is not i32 or
            lam.dtype is not names.f32 or out.get_device() != dev or
            k_cache.get_device() != dev or v_cache.get_device() != dev or
            block_tables.get_device() != dev or seq_lens.get_device() != dev or
            lam.get_device() != dev or
            not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and
                 v_cache.is_contiguous() and block_tables.is_contiguous() and
                 seq_lens.is_contiguous() and lam.is_contiguous())):
        raise ValueError(_NEAR)
    w = 0 if norm_weight is None else _weights(norm_weight, shape[2], dt, dev)
    return dev, (out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                 block_tables.data_ptr(), seq_lens.data_ptr()), (lam.data_ptr(), w)


def _bytes_of(workspace, dev):
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous, on the current CUDA device")
    return workspace.nbytes


def diff_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                               max_blocks_per_seq) -> int:
    return int(load().pa_diff_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                    max_blocks_per_seq))


def diff_decode_workspace_for(q, k_cache, block_tables, stream=None):
    """A workspace tensor sized for pa_diff_decode on these shapes."""
    n, hq, d = q.shape
    nbytes = diff_decode_workspace_size(n, hq, k_cache.shape[1], d, block_tables.shape[1])
    return _scratch(nbytes, q.device, stream) if nbytes else None


def diff_decode(out, q, k_cache, v_cache, block_tables, seq_lens, lam, scale, norm_weight=None,
                eps=1e-6, out_scale=1.0, workspace=None, stream=None):
    """pa_diff_decode: differential attention of one query token per sequence.

    q, out [num_seqs, num_heads, head_dim], a head's row holding its two
    queries; the pools of decode, a key row holding the two keys; lam float32
    [num_heads] weighs the second map.  With norm_weight [head_dim] the result is
    RMS-normalised over the head, and it is multiplied by out_scale either way.
    """
    n, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    if seq_lens.shape != (n,):
        raise ValueError("shapes")
    names = _hot()
    dev, at, factors = _diff_pointers(out, q, k_cache, v_cache, block_tables, seq_lens, lam,
                                      norm_weight, names)
    if workspace is None:
        workspace = diff_decode_workspace_for(q, k_cache, block_tables, stream)
    wptr, wbytes = ((0, 0) if workspace is None else
                    (workspace.data_ptr(), _bytes_of(workspace, dev)))
    rc = load().pa_diff_decode_args(_DIFF_ARGS.pack(
        _DIFF_ARGS.size, *at, 0, *factors, wptr,
        names.raw_stream(dev) if stream is None else stream.cuda_stream, wbytes, scale, eps,
        out_scale, n, 0, hq, hkv, d, bs, block_tables.shape[1], nb, _code(q.dtype, names)))
    if rc:
        raise PagedAttnError("pa_diff_decode", rc)
    return out


def diff_prefill_workspace_size(num_seqs, max_query_len, num_heads, num_kv_heads) -> int:
    return int(load().pa_diff_prefill_workspace_size(num_seqs, max_query_len, num_heads,
                                                     num_kv_heads))


def diff_prefill_workspace_for(q, k_cache, seq_lens, max_query_len, stream=None):
    """A workspace tensor sized for pa_diff_prefill on these shapes."""
    nbytes = diff_prefill_workspace_size(seq_lens.shape[0], int(max_query_len), q.shape[1],
                                         k_cache.shape[1])
    return _scratch(nbytes, q.device, stream) if nbytes else None


def diff_prefill(out, q, k_cache, v_cache, block_tables, seq_lens, query_start, max_query_len, lam,
                 scale, norm_weight=None, eps=1e-6, out_scale=1.0, workspace="auto", stream=None):
    """pa_diff_prefill: differential attention of each sequence's newest chunk, causal.

    Rows, tables, query_start, max_query_len and workspace as prefill; lam,
    norm_weight, eps and out_scale as diff_decode.
    """
    t, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    n, longest = seq_lens.shape[0], int(max_query_len)
    if query_start.shape != (n + 1,):
        raise ValueError("shapes")
    names = _hot()
    dev, at, factors = _diff_pointers(out, q, k_cache, v_cache, block_tables, seq_lens, lam,
                                      norm_weight, names)
    if isinstance(workspace, str):
        workspace = diff_prefill_workspace_for(q, k_cache, seq_lens, longest, stream)
    wptr, wbytes = ((0, 0) if workspace is None else
                    (workspace.data_ptr(), _bytes_of(workspace, dev)))
    rc = load().pa_diff_prefill_args(_DIFF_ARGS.pack(
        _DIFF_ARGS.size, *at, _near(query_start, names.i32, dev), *factors, wptr,
        names.raw_stream(dev) if stream is None else stream.cuda_stream, wbytes, scale, eps,
        out_scale, n, longest, hq, hkv, d, bs, block_tables.shape[1], nb, _code(q.dtype, names)))
    if rc:
        raise PagedAttnError("pa_diff_prefill", rc)
    return out


def decode_noalloc(out, q, k_cache, v_cache, block_tables, seq_lens, scale, stream=None):
    """pa_decode_noalloc: decode with the library's own fixed scratch (balanced split).

    For callers that cannot allocate a workspace.  Calls share one scratch
    array per device, so calls that may overlap on the GPU must be ordered on
    one stream; the first call on a device must come before any stream capture.
    """
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _require(out.shape == q.shape and d2 == d and v_cache.shape == k_cache.shape, "shapes")
    _require(block_tables.dim() == 2 and block_tables.shape[0] == n and seq_lens.shape == (n,),
             "table shapes")
    rc = load().pa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(block_tables), _ptr(seq_lens), n, hq, hkv, d, bs,
                                  block_tables.shape[1], nb, float(scale), _dtype_code(q),
                                  _stream(stream))
    _check("pa_decode_noalloc", rc)
    return out


def reshape_and_cache(k_new, v_new, k_cache, v_cache, slot_mapping, stream=None):
    """pa_reshape_and_cache: write token i's K/V into pool slot slot_mapping[i] (<0 skips)."""
    nt, hkv, d = k_new.shape
    nb, hkv2, bs, d2 = k_cache.shape
    _require(hkv == hkv2 and d == d2 and v_new.shape == k_new.shape, "shapes")
    _require(slot_mapping.shape == (nt,), "slot_mapping shape")
    rc = load().pa_reshape_and_cache(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(slot_mapping), nt, hkv, d, bs, nb, _dtype_code(k_cache),
                                     _stream(stream))
    _check("pa_reshape_and_cache", rc)


def _rows(t, shape, dtype, device):
    """Elements between the tokens of [tokens, heads, head_dim] rows whose heads lie
    one after the other (any distance between tokens: slices of a projection's output)."""
    n, h, d = shape
    st, sh, se = t.stride()
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != device or se != 1 or
            (sh != d and h != 1)):
        raise ValueError(f"rows: {tuple(shape)} of {dtype} on device {device}, a token's heads "
                         "one after the other")
    return st if n > 1 else h * d


def rope_and_cache(q_out, q, k_new, v_new, k_cache, v_cache, slot_mapping, positions, cos_sin,
                   q_norm=None, k_norm=None, eps=1e-6, interleaved=False, num_maps=1, stream=None):
    """pa_rope_and_cache: q and k normalised per head (with q_norm, k_norm) and rotated
    by their positions; q goes to q_out, k and v into pool slot slot_mapping[i].

    q, q_out [tokens, heads, head_dim]; k_new, v_new [tokens, kv_heads, head_dim];
    tokens may lie any distance apart (slices of one projection's output), and
    q_out may be q.  slot_mapping int64 and positions int32 [tokens], negative for
    padding; cos_sin float32 [max_position, rotary_dim], each row the cosines, then
    the sines, of its position's rotary_dim / 2 angles, for example
        a = torch.arange(max_position).double()[:, None] * inv_freq[None]
        cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
    num_maps=2 treats a head as two keys of half its size (differential attention).
    """
    names = _hot()
    n, hq, d = q_shape = q.shape
    nb, hkv, bs, d2 = pool = k_cache.shape
    table, rot = cos_sin.shape
    new = (n, hkv, d)
    dt, dev, num_maps = q.dtype, _current(q, names), int(num_maps)
    if d2 != d or v_cache.shape != pool or positions.shape != (n,) or slot_mapping.shape != (n,):
        raise ValueError("shapes")
    if (k_cache.dtype is not dt or v_cache.dtype is not dt or
            slot_mapping.dtype is not names.i64 or positions.dtype is not names.i32 or
            cos_sin.dtype is not names.f32 or k_cache.get_device() != dev or
            v_cache.get_device() != dev or slot_mapping.get_device() != dev or
            positions.get_device() != dev or cos_sin.get_device() != dev or
            not (k_cache.is_contiguous() and v_cache.is_contiguous() and
                 slot_mapping.is_contiguous() and positions.is_contiguous() and
                 cos_sin.is_contiguous())):
        raise ValueError(_NEAR)
    seg = d // num_maps if num_maps > 0 else 0
    qw = 0 if q_norm is None else _weights(q_norm, seg, dt, dev)
    kw = 0 if k_norm is None else _weights(k_norm, seg, dt, dev)
    rc = load().pa_rope_and_cache_args(_ROPE_ARGS.pack(
        _ROPE_ARGS.size, q_out.data_ptr(), 0, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(),
        cos_sin.data_ptr(), qw, kw, names.raw_stream(dev) if stream is None else stream.cuda_stream,
        _rows(q, q_shape, dt, dev), _rows(k_new, new, dt, dev), _rows(v_new, new, dt, dev),
        _rows(q_out, q_shape, dt, dev), 0, eps, n, hq, hkv, d, num_maps, bs, nb, table, rot,
        1 if interleaved else 0, _code(dt, names)))
    if rc:
        raise PagedAttnError("pa_rope_and_cache", rc)
    return q_out


def qk_norm_rope(q_out, k_out, q, k, positions, cos_sin, q_norm=None, k_norm=None, eps=1e-6,
                 interleaved=False, num_maps=1, stream=None):
    """pa_qk_norm_rope: rope_and_cache's normalisation and rotation without the pool, for
    decode_append and decode_shared_prefix, which write the new tokens themselves.
    q_out may be q and k_out may be k."""
    names = _hot()
    n, hq, d = q_shape = q.shape
    hkv = k.shape[1]
    table, rot = cos_sin.shape
    new = (n, hkv, d)
    dt, dev, num_maps = q.dtype, _current(q, names), int(num_maps)
    if positions.shape != (n,):
        raise ValueError("shapes")
    if (positions.dtype is not names.i32 or cos_sin.dtype is not names.f32 or
            positions.get_device() != dev or cos_sin.get_device() != dev or
            not (positions.is_contiguous() and cos_sin.is_contiguous())):
        raise ValueError(_NEAR)
    seg = d // num_maps if num_maps > 0 else 0
    qw = 0 if q_norm is None else _weights(q_norm, seg, dt, dev)
    kw = 0 if k_norm is None else _weights(k_norm, seg, dt, dev)
    rc = load().pa_qk_norm_rope_args(_ROPE_ARGS.pack(
        _ROPE_ARGS.size, q_out.data_ptr(), k_out.data_ptr(), q.data_ptr(), k.data_ptr(), 0, 0, 0, 0,
        positions.data_ptr(), cos_sin.data_ptr(), qw, kw,
        names.raw_stream(dev) if stream is None else stream.cuda_stream,
        _rows(q, q_shape, dt, dev), _rows(k, new, dt, dev), 0, _rows(q_out, q_shape, dt, dev),
        _rows(k_out, new, dt, dev), eps, n, hq, hkv, d, num_maps, 0, 0, table, rot,
        1 if interleaved else 0, _code(dt, names)))
    if rc:
        raise PagedAttnError("pa_qk_norm_rope", rc)
    return q_out, k_out


def copy_blocks(k_cache, v_cache, block_mapping, stream=None):
    """pa_copy_blocks: whole-block copies src -> dst for each row of block_mapping [P, 2]."""
    nb, hkv, bs, d = k_cache.shape
    _require(block_mapping.dim() == 2 and block_mapping.shape[1] == 2, "block_mapping shape")
    rc = load().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_mapping),
                               block_mapping.shape[0], hkv, d, bs, nb, _dtype_code(k_cache),
                               _stream(stream))
    _check("pa_copy_blocks", rc)


def swap_blocks(dst_k, dst_v, src_k, src_v, block_mapping, stream=None):
    """pa_swap_blocks: whole-block copies src -> dst between two pools (one of them
    typically in page-locked host memory, e.g. ``torch.empty(..).pin_memory()``)."""
    snb, hkv, bs, d = src_k.shape
    dnb = dst_k.shape[0]
    _require(dst_k.shape[1:] == src_k.shape[1:] and dst_v.shape == dst_k.shape and
             src_v.shape == src_k.shape, "pool shapes")
    _require(block_mapping.dim() == 2 and block_mapping.shape[1] == 2, "block_mapping shape")
    rc = load().pa_swap_blocks(_ptr(dst_k), _ptr(dst_v), _ptr(src_k), _ptr(src_v),
                               _ptr(block_mapping), block_mapping.shape[0], hkv, d, bs, snb, dnb,
                               _dtype_code(src_k), _stream(stream))
    _check("pa_swap_blocks", rc)


def gather_kv(k_out, v_out, k_cache, v_cache, block_tables, seq_lens, stream=None):
    """pa_gather_kv: k_out[s, h, t] = k_cache[table[s][t//16], h, t%16] for t < seq_lens[s]."""
    nb, hkv, bs, d = k_cache.shape
    n, mb = block_tables.shape
    _require(k_out.shape == (n, hkv, mb * bs, d) and v_out.shape == k_out.shape, "out shape")
    rc = load().pa_gather_kv(_ptr(k_out), _ptr(v_out), _ptr(k_cache), _ptr(v_cache),
                             _ptr(block_tables), _ptr(seq_lens), n, hkv, d, bs, mb, nb,
                             _dtype_code(k_cache), _stream(stream))
    _check("pa_gather_kv", rc)


def validate_tables(block_tables, seq_lens, num_blocks, bad_count, stream=None):
    """pa_validate_tables: adds to bad_count (uint32/int32 device scalar) the bad entries."""
    n, mb = block_tables.shape
    rc = load().pa_validate_tables(_ptr(block_tables), _ptr(seq_lens), n, mb, num_blocks,
                                   BLOCK_SIZE, _ptr(bad_count), _stream(stream))
    _check("pa_validate_tables", rc)


def selftest_bounded_wait(limit_us=2000, stream=None):
    """pa_selftest_bounded_wait: a copy wait that must time out and report it."""
    _check("pa_selftest_bounded_wait", load().pa_selftest_bounded_wait(int(limit_us),
                                                                       _stream(stream)))


def get_device_error(clear=True, stream=None) -> int:
    """Synchronise and return (and by default clear) the PA_DEVERR_* bits."""
    bits = C.c_uint32(0)
    rc = load().pa_get_device_error(_stream(stream), C.byref(bits), 1 if clear else 0)
    if rc not in (0, 5):
        _check("pa_get_device_error", rc)
    return int(bits.value)
