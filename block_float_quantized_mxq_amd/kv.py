"""Binding of include/mxq_kv.h: rotary positions, the paged key/value cache and
attention over it.  Argument marshalling only, as in the rest of the package;
every name here is exported by the package itself.

Tensors:
  q, k, v       [tokens, heads, head_dim], float32 or bfloat16; rows may be strided (slices of a fused QKV row),
                the heads of a token may not
  cache         KVCache: k, v [pages, kv_heads, page_size, head_dim] bfloat16, or uint8 E4M3 codes with
                uint8 E8M0 scales [..., head_dim / 32]
  block_table   int32 [seqs, max_pages]; rows may be strided
  cu_q          int32 [seqs + 1]: sequence s owns rows cu_q[s] .. cu_q[s + 1] of q, k and v
  kv_lens       int32 [seqs]: cached positions of a sequence, its new tokens included

A call runs on the device of its tensors, on that device's current stream or the one given.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

KV_BF16, KV_MXFP8 = 0, 2
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int64), ("layout", ctypes.c_int32),
                ("mscale", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("reserved", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64)]


class _Seqs(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64)]


def bind(L):
    """Argument types of the entry points of include/mxq_kv.h on the loaded library."""
    P, I64, I, F, D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_double
    L.mxq_rope_inv_freq.argtypes = [I, I64, D, D, D, D, D, P, P]
    L.mxq_rope.argtypes = [P, I, P, I, P, P, I64, I64, I64, I64, I64, P]
    L.mxq_kv_append.argtypes = [P, P, P, I, P, P, P, P, P, I64, I64, I64, I64, I64, P]
    L.mxq_paged_attn.argtypes = [P, P, P, P, P, I64, I64, I64, F, I64, I64, P, I64, P]
    L.mxq_paged_attn_workspace.argtypes = [P, P, I64, I64, I64]
    L.mxq_paged_attn_workspace.restype = I64
    for f in (L.mxq_rope_inv_freq, L.mxq_rope, L.mxq_kv_append, L.mxq_paged_attn, L.mxq_kv_version):
        f.restype = I


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import lib
        _loaded = lib()
    return _loaded


def _check(st, what):
    if st != 0:
        from . import MxqError
        raise MxqError(st, what)


_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
_X = (_F32, _BF16)
_Tensor = torch.Tensor


# The checks run before every launch, so they are written for the case that passes; _refuse says what was wrong.
def _refuse(t, dtypes, name, index):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, the call's other tensors are on cuda:{index}")


def _first(t, dtypes, name):
    """The device index of the tensor that decides where a call runs."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dtype not in dtypes:
        _refuse(t, dtypes, name, -1)
    return t.get_device()


def _flat(t, dtype, name, index, shape):
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, (dtype,), name, index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _heads_of(t, dtypes, name, index):
    """[tokens, heads, dim] whose heads are adjacent; returns the tokens' stride in elements."""
    if not isinstance(t, _Tensor) or t.dtype not in dtypes or t.get_device() != index:
        _refuse(t, dtypes, name, index)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    n, h, d = t.shape
    stride, head, elem = t.stride()
    if (d > 1 and elem != 1) or (h > 1 and head != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return stride if n > 1 else h * d


@contextlib.contextmanager
def _guard(index, stream):
    with torch.cuda.device(index):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_HERE = contextlib.nullcontext()


def _on(index, stream):
    """Context in which allocations belong to the call's stream and the call's device is the current one."""
    if stream is None and _current_device() == index:
        return _HERE
    if stream is not None and stream.device_index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{index}")
    return _guard(index, stream)


# torch's own shortcuts to the current device and stream, without the objects that torch.cuda builds around them
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)


def _raw_stream(index, stream):
    return _current_raw_stream(index) if stream is None else stream.cuda_stream


def _layout(layout):
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    return ROPE_LAYOUTS[layout]


def _rope_params(inv_freq, layout, mscale, index):
    code = _layout(layout)
    if inv_freq is None:
        return _Rope(None, 0, code, 1.0)
    p = _flat(inv_freq, _F32, "inv_freq", index, (inv_freq.numel() if isinstance(inv_freq, _Tensor) else 0,))
    return _Rope(p, 2 * inv_freq.numel(), code, mscale)


class KVCache:
    """A paged cache over the caller's tensors, made once and kept: k, v [pages, kv_heads, page_size, head_dim] in
    bfloat16, or uint8 E4M3 codes with uint8 E8M0 scales k_scales, v_scales [pages, kv_heads, page_size,
    head_dim / 32]."""

    __slots__ = ("_tensors", "device", "shape", "format", "_index", "_c", "_ref", "__weakref__")

    def __init__(self, k, v, k_scales=None, v_scales=None):
        mx = k_scales is not None or v_scales is not None
        dtype = _U8 if mx else _BF16
        index = _first(k, (dtype,), "cache k")
        if k.dim() != 4:
            raise ValueError("cache k must be [pages, kv_heads, page_size, head_dim]")
        shape = k.shape
        pages, heads, page, dim = shape
        kp, vp = _flat(k, dtype, "cache k", index, shape), _flat(v, dtype, "cache v", index, shape)
        ks = vs = None
        if mx:
            if dim % 32:
                raise ValueError(f"head_dim {dim} is not a multiple of the MXFP8 block of 32")
            want = (pages, heads, page, dim // 32)
            ks = _flat(k_scales, _U8, "cache k_scales", index, want)
            vs = _flat(v_scales, _U8, "cache v_scales", index, want)
        self._tensors = (k, v, k_scales, v_scales)
        self.device, self.shape, self.format = k.device, shape, KV_MXFP8 if mx else KV_BF16
        self._index = index
        self._c = _Cache(self.format, 0, kp, vp, ks, vs, pages, page, heads, dim)
        self._ref = ctypes.byref(self._c)

    # read-only: the addresses were taken when the cache was made
    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scales = property(lambda self: self._tensors[2])
    v_scales = property(lambda self: self._tensors[3])


def kv_cache(pages, kv_heads, page_size, head_dim, fmt="bf16", device="cuda"):
    """A zeroed KVCache; fmt "bf16" or "mxfp8"."""
    shape = (pages, kv_heads, page_size, head_dim)
    if fmt == "bf16":
        return KVCache(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
    if fmt != "mxfp8":
        raise ValueError(f"fmt must be 'bf16' or 'mxfp8', got {fmt!r}")
    parts = [torch.zeros(s, dtype=torch.uint8, device=device)
             for s in (shape, shape, (*shape[:3], head_dim // 32), (*shape[:3], head_dim // 32))]
    return KVCache(*parts)


def _seqs_of(index, block_table, cu_q, kv_lens):
    if not isinstance(block_table, _Tensor) or block_table.dtype is not _I32 or block_table.get_device() != index:
        _refuse(block_table, (_I32,), "block_table", index)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [seqs, max_pages]")
    seqs, width = block_table.shape
    stride, elem = block_table.stride()
    if width > 1 and elem != 1:
        raise ValueError("the rows of block_table must be contiguous")
    return _Seqs(block_table.data_ptr(), _flat(cu_q, _I32, "cu_q", index, (seqs + 1,)),
                 _flat(kv_lens, _I32, "kv_lens", index, (seqs,)), seqs, width, stride if seqs > 1 else width)


def rope_inv_freq(rot_dim, theta=10000.0, scaling=None, factor=1.0, context=0, low=1.0, high=32.0, device="cuda"):
    """(inv_freq float32 [rot_dim / 2] on the device, mscale) of a rotation: scaling None, "linear", "ntk", "yarn"
    or "bands" (see mxq_rope_inv_freq; context, low and high are for the last two)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALINGS)[1:]} or None, got {scaling!r}")
    table = (ctypes.c_float * max(1, rot_dim // 2))()
    mscale = ctypes.c_float()
    _check(_lib().mxq_rope_inv_freq(ROPE_SCALINGS[scaling], rot_dim, theta, factor, context, low, high,
                                    ctypes.cast(table, ctypes.c_void_p), ctypes.addressof(mscale)),
           "mxq_rope_inv_freq")
    return torch.tensor(list(table), dtype=torch.float32).to(device), float(mscale.value)


def rope(x, positions, inv_freq, layout="half", mscale=1.0, out=None, out_dtype=torch.bfloat16, stream=None):
    """Rotary positions of x [tokens, heads, head_dim] (float32 or bfloat16) -> out_dtype (float32 or bfloat16),
    same shape.  positions int32 [tokens]; the first 2 * len(inv_freq) elements of a head turn.  out may be x
    (in place) if the types agree, else it must not overlap x."""
    index = _first(x, _X, "x")
    xs = _heads_of(x, _X, "x", index)
    n, h, d = x.shape
    pos = _flat(positions, _I32, "positions", index, (n,))
    r = _rope_params(inv_freq, layout, mscale, index)
    if out is not None:
        _first(out, _X, "out")
        out_dtype = out.dtype
    if out_dtype not in _X:
        raise TypeError(f"out must be float32 or bfloat16, got {out_dtype}")
    with _on(index, stream):
        if out is None:
            out, ys = torch.empty((n, h, d), dtype=out_dtype, device=x.device), h * d
        else:
            ys = _heads_of(out, _X, "out", index)
            if out.shape != x.shape:
                raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
        _check(_lib().mxq_rope(x.data_ptr(), x.dtype is _BF16, out.data_ptr(), out_dtype is _BF16, pos, ctypes.byref(r),
                               n, h, d, xs, ys, _raw_stream(index, stream)), "mxq_rope")
    return out


def kv_append(k, v, cache, block_table, cu_q, kv_lens, q=None, inv_freq=None, layout="half", mscale=1.0,
              positions=None, q_out=None, stream=None):
    """Appends the new tokens' keys (rotated) and values [tokens, kv_heads, head_dim] to the cache; with q
    [tokens, heads, head_dim] also returns the rotated queries, bfloat16 (else None).  k, v and q share one type,
    float32 or bfloat16.  inv_freq None: nothing turns.  positions int32 [tokens]: what to rotate by (default: the
    tokens' positions in the cache).  Rows outside every sequence are left as they were: in q_out too, which is
    allocated uninitialised when None."""
    index = cache._index
    ks = _heads_of(k, _X, "k", index)
    same = (k.dtype,)
    vs = _heads_of(v, same, "v", index)
    n, hk, d = k.shape
    if v.shape != k.shape or hk != cache._c.kv_heads or d != cache._c.head_dim:
        raise ValueError(f"k {tuple(k.shape)}, v {tuple(v.shape)} and the cache {tuple(cache.shape)} disagree")
    qs, h, qp, op, pp = 0, hk, None, None, None
    if q is not None:
        qs = _heads_of(q, same, "q", index)
        h, qp = q.shape[1], q.data_ptr()
        if q.shape[0] != n or q.shape[2] != d:
            raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    r = _rope_params(inv_freq, layout, mscale, index)
    if positions is not None:
        pp = _flat(positions, _I32, "positions", index, (n,))
    s = _seqs_of(index, block_table, cu_q, kv_lens)
    with _on(index, stream):
        if q is not None:
            if q_out is None:
                q_out = torch.empty((n, h, d), dtype=_BF16, device=cache.device)
                op = q_out.data_ptr()
            else:
                op = _flat(q_out, _BF16, "q_out", index, (n, h, d))
        _check(_lib().mxq_kv_append(qp, k.data_ptr(), v.data_ptr(), k.dtype is _BF16, op, pp, ctypes.byref(r), cache._ref,
                                    ctypes.byref(s), n, h, qs, ks, vs, _raw_stream(index, stream)), "mxq_kv_append")
    return q_out


def paged_attn_workspace(cache, block_table, cu_q, kv_lens, tokens, heads, max_q):
    """Bytes of workspace that paged_attn uses for these sizes."""
    s = _seqs_of(cache._index, block_table, cu_q, kv_lens)
    size = _lib().mxq_paged_attn_workspace(cache._ref, ctypes.byref(s), tokens, heads, max_q)
    if size < 0:
        raise ValueError(f"no paged_attn of {tokens} tokens and {heads} heads with max_q {max_q} over {tuple(cache.shape)}")
    return size


def paged_attn(q, cache, block_table, cu_q, kv_lens, scale=None, window=0, max_q=None, out=None, lse=None,
               workspace=None, stream=None):
    """Attention of the new tokens' queries q bfloat16 [tokens, heads, head_dim] over the cache, which already
    holds their keys and values -> bfloat16 [tokens, heads, head_dim].  A token at position p sees positions
    j <= p, and j > p - window if window > 0.  scale defaults to head_dim ** -0.5; max_q (default: all the
    tokens) is a hint, the largest number of new tokens of a sequence; lse: float32 [tokens, heads] to receive
    the log-sum-exp; workspace: uint8, at least paged_attn_workspace bytes (allocated when None).  Rows outside
    every sequence are left as they were (in an `out` allocated here: uninitialised)."""
    index = cache._index
    qs = _heads_of(q, (_BF16,), "q", index)
    n, h, d = q.shape
    if d != cache._c.head_dim:
        raise ValueError(f"q {tuple(q.shape)} and the cache {tuple(cache.shape)} disagree")
    s = _seqs_of(index, block_table, cu_q, kv_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    if max_q is None:
        max_q = n
    L = _lib()
    sp = ctypes.byref(s)
    lp = None if lse is None else _flat(lse, _F32, "lse", index, (n, h))
    wp, size = None, 0
    with _on(index, stream):
        if out is None:
            out = torch.empty((n, h, d), dtype=_BF16, device=cache.device)
            op = out.data_ptr()
        else:
            op = _flat(out, _BF16, "out", index, (n, h, d))
        if workspace is None:
            size = L.mxq_paged_attn_workspace(cache._ref, sp, n, h, max_q)
            if size > 0:
                workspace = torch.empty((size,), dtype=_U8, device=cache.device)
                wp = workspace.data_ptr()
            size = max(size, 0)
        else:
            size = workspace.numel() if isinstance(workspace, _Tensor) else 0
            wp = _flat(workspace, _U8, "workspace", index, (size,))
        _check(L.mxq_paged_attn(q.data_ptr(), op, lp, cache._ref, sp, n, h, qs, scale, window, max_q, wp, size,
                                _raw_stream(index, stream)), "mxq_paged_attn")
    return out
