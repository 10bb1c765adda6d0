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


def _lib():
    from . import lib
    return lib()


def _check(st, what):
    if st != 0:
        from . import MxqError
        raise MxqError(st, what)


def _need(t, dtypes, name, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors are on {device}")
    return t


def _flat(t, dtypes, name, device, shape=None):
    _need(t, dtypes, name, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


_X = (torch.float32, torch.bfloat16)
_BF16, _F32, _I32, _U8 = (torch.bfloat16,), (torch.float32,), (torch.int32,), (torch.uint8,)


def _heads_of(t, dtypes, name, device=None):
    """[tokens, heads, dim] whose heads are adjacent; returns the tokens' stride in elements."""
    _need(t, dtypes, name, device)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    n, h, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return t.stride(0) if n > 1 else h * d


@contextlib.contextmanager
def _guard(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _on(device, stream):
    """Context in which allocations belong to the call's stream and the call's device is the current one."""
    if stream is None and torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    return _guard(device, stream)


def _raw_stream(device, stream):
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _layout(layout):
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    return ROPE_LAYOUTS[layout]


def _rope_params(inv_freq, layout, mscale, device):
    code = _layout(layout)
    if inv_freq is None:
        return _Rope(None, 0, code, 1.0)
    _flat(inv_freq, _F32, "inv_freq", device)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must have one dimension")
    return _Rope(inv_freq.data_ptr(), 2 * inv_freq.numel(), code, mscale)


class KVCache:
    """A paged cache over the caller's tensors: k, v [pages, kv_heads, page_size, head_dim] in bfloat16, or uint8
    E4M3 codes with uint8 E8M0 scales k_scales, v_scales [pages, kv_heads, page_size, head_dim / 32]."""

    __slots__ = ("k", "v", "k_scales", "v_scales", "device", "shape", "format", "_c")

    def __init__(self, k, v, k_scales=None, v_scales=None):
        mx = k_scales is not None or v_scales is not None
        _need(k, _U8 if mx else _BF16, "cache k")
        if k.dim() != 4:
            raise ValueError("cache k must be [pages, kv_heads, page_size, head_dim]")
        shape = k.shape
        _flat(k, _U8 if mx else _BF16, "cache k", None)
        _flat(v, _U8 if mx else _BF16, "cache v", k.device, shape)
        if mx:
            if shape[3] % 32:
                raise ValueError(f"head_dim {shape[3]} is not a multiple of the MXFP8 block of 32")
            want = (*shape[:3], shape[3] // 32)
            _flat(k_scales, _U8, "cache k_scales", k.device, want)
            _flat(v_scales, _U8, "cache v_scales", k.device, want)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.device, self.shape, self.format = k.device, tuple(shape), KV_MXFP8 if mx else KV_BF16
        self._c = _Cache(self.format, 0, k.data_ptr(), v.data_ptr(), k_scales.data_ptr() if mx else None,
                         v_scales.data_ptr() if mx else None, shape[0], shape[2], shape[1], shape[3])


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


def _seqs_of(cache, block_table, cu_q, kv_lens):
    _need(block_table, _I32, "block_table", cache.device)
    if block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [seqs, max_pages] with contiguous rows")
    seqs, width = block_table.shape
    _flat(cu_q, _I32, "cu_q", cache.device, (seqs + 1,))
    _flat(kv_lens, _I32, "kv_lens", cache.device, (seqs,))
    return _Seqs(block_table.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(), seqs, width,
                 block_table.stride(0) if seqs > 1 else width)


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
    xs = _heads_of(x, _X, "x")
    dev = x.device
    n, h, d = x.shape
    _flat(positions, _I32, "positions", dev, (n,))
    r = _rope_params(inv_freq, layout, mscale, dev)
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _X:
        raise TypeError(f"out must be float32 or bfloat16, got {out_dtype}")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((n, h, d), dtype=out_dtype, device=dev)
        ys = _heads_of(out, _X, "out", dev)
        if out.shape != x.shape:
            raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
        _check(_lib().mxq_rope(x.data_ptr(), x.dtype == torch.bfloat16, out.data_ptr(), out_dtype == torch.bfloat16,
                               positions.data_ptr(), ctypes.byref(r), n, h, d, xs, ys, _raw_stream(dev, stream)),
               "mxq_rope")
    return out


def kv_append(k, v, cache, block_table, cu_q, kv_lens, q=None, inv_freq=None, layout="half", mscale=1.0,
              positions=None, q_out=None, stream=None):
    """Appends the new tokens' keys (rotated) and values [tokens, kv_heads, head_dim] to the cache; with q
    [tokens, heads, head_dim] also returns the rotated queries, bfloat16 (else None).  k, v and q share one type,
    float32 or bfloat16.  inv_freq None: nothing turns.  positions int32 [tokens]: what to rotate by (default: the
    tokens' positions in the cache).  Rows outside every sequence are left as they were: in q_out too, which is
    allocated uninitialised when None."""
    ks = _heads_of(k, _X, "k", cache.device)
    vs = _heads_of(v, (k.dtype,), "v", cache.device)
    dev = cache.device
    n, hk, d = k.shape
    if v.shape != k.shape or (hk, d) != (cache.shape[1], cache.shape[3]):
        raise ValueError(f"k {tuple(k.shape)}, v {tuple(v.shape)} and the cache {cache.shape} disagree")
    qs, h = 0, hk
    if q is not None:
        qs = _heads_of(q, (k.dtype,), "q", dev)
        h = q.shape[1]
        if q.shape[0] != n or q.shape[2] != d:
            raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    r = _rope_params(inv_freq, layout, mscale, dev)
    if positions is not None:
        _flat(positions, _I32, "positions", dev, (n,))
    s = _seqs_of(cache, block_table, cu_q, kv_lens)
    with _on(dev, stream):
        if q is not None:
            if q_out is None:
                q_out = torch.empty((n, h, d), dtype=torch.bfloat16, device=dev)
            _flat(q_out, _BF16, "q_out", dev, (n, h, d))
        _check(_lib().mxq_kv_append(None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                    k.dtype == torch.bfloat16, None if q is None else q_out.data_ptr(),
                                    None if positions is None else positions.data_ptr(), ctypes.byref(r),
                                    ctypes.byref(cache._c), ctypes.byref(s), n, h, qs, ks, vs,
                                    _raw_stream(dev, stream)), "mxq_kv_append")
    return q_out


def paged_attn_workspace(cache, block_table, cu_q, kv_lens, tokens, heads, max_q):
    """Bytes of workspace that paged_attn uses for these sizes."""
    s = _seqs_of(cache, block_table, cu_q, kv_lens)
    return _lib().mxq_paged_attn_workspace(ctypes.byref(cache._c), ctypes.byref(s), tokens, heads, max_q)


def paged_attn(q, cache, block_table, cu_q, kv_lens, scale=None, window=0, max_q=None, out=None, lse=None,
               workspace=None, stream=None):
    """Attention of the new tokens' queries q bfloat16 [tokens, heads, head_dim] over the cache, which already
    holds their keys and values -> bfloat16 [tokens, heads, head_dim].  A token at position p sees positions
    j <= p, and j > p - window if window > 0.  scale defaults to head_dim ** -0.5; max_q (default: all the
    tokens) is a hint, the largest number of new tokens of a sequence; lse: float32 [tokens, heads] to receive
    the log-sum-exp; workspace: uint8, at least paged_attn_workspace bytes (allocated when None).  Rows outside
    every sequence are left as they were (in an `out` allocated here: uninitialised)."""
    qs = _heads_of(q, _BF16, "q", cache.device)
    dev = cache.device
    n, h, d = q.shape
    if d != cache.shape[3]:
        raise ValueError(f"q {tuple(q.shape)} and the cache {cache.shape} disagree")
    s = _seqs_of(cache, block_table, cu_q, kv_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    if max_q is None:
        max_q = n
    L = _lib()
    c, sp = ctypes.byref(cache._c), ctypes.byref(s)
    if lse is not None:
        _flat(lse, _F32, "lse", dev, (n, h))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((n, h, d), dtype=torch.bfloat16, device=dev)
        else:
            _flat(out, _BF16, "out", dev, (n, h, d))
        if workspace is None:
            need = L.mxq_paged_attn_workspace(c, sp, n, h, max_q)
            if need > 0:
                workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
        else:
            _flat(workspace, _U8, "workspace", dev)
        _check(L.mxq_paged_attn(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), c, sp, n, h,
                                qs, scale, window, max_q, None if workspace is None else workspace.data_ptr(),
                                0 if workspace is None else workspace.numel(), _raw_stream(dev, stream)),
               "mxq_paged_attn")
    return out
