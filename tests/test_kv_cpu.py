"""The positions-and-cache entry points without a GPU: every refusal (validation runs before any HIP call, so the
bogus-but-aligned pointers are never touched), the header, and the inverse frequencies."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import block_float_quantized_mxq_amd as mxq
from block_float_quantized_mxq_amd import kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLPTR, SHAPE, ALIGN, FORMAT, UNSUPPORTED, DEVICE = 0, 1, 2, 3, 4, 5, 6
A = 0x10000


def test_header_and_exports():
    text = open(os.path.join(ROOT, "include", "mxq_kv.h")).read()
    declared = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(mxq_\w+)\s*\(", text, re.M)))
    assert declared == ["mxq_kv_append", "mxq_kv_version", "mxq_paged_attn", "mxq_paged_attn_workspace", "mxq_rope",
                        "mxq_rope_inv_freq"]
    out = subprocess.run(["nm", "-D", "--defined-only", mxq.LIB_PATH], capture_output=True, text=True, check=True).stdout
    for name in declared:
        assert re.search(rf"\b{name}\b", out), name
    assert mxq.lib().mxq_kv_version() == 1


def test_header_compiles_as_c_and_matches_the_binding():
    src = '#include "mxq_kv.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu", sizeof(mxq_rope_params_t), ' \
          'sizeof(mxq_kv_cache_t), sizeof(mxq_kv_seqs_t)); return 0; }'
    exe = os.path.join(ROOT, "_build", "kv_header_check")
    os.makedirs(os.path.dirname(exe), exist_ok=True)
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-x", "c", "-", "-o", exe],
                   input=src, text=True, check=True)
    sizes = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(s) for s in sizes] == [ctypes.sizeof(t) for t in (kv._Rope, kv._Cache, kv._Seqs)]


def rope(x=A, xt=0, y=2 * A, yt=1, pos=A, inv=A, rot=64, layout=0, null_rope=False, tokens=3, heads=4, dim=64, xs=256,
         ys=256):
    r = kv._Rope(inv, rot, layout, 1.0)
    return mxq.lib().mxq_rope(x, xt, y, yt, pos, None if null_rope else ctypes.byref(r), tokens, heads, dim, xs, ys, None)


def cache_struct(fmt=0, reserved=0, k=A, v=A, ks=None, vs=None, pages=4, page=16, hk=2, dim=64):
    return kv._Cache(fmt, reserved, k, v, ks, vs, pages, page, hk, dim)


def seqs_struct(table=A, cu=A, lens=A, seqs=2, width=3, stride=3):
    return kv._Seqs(table, cu, lens, seqs, width, stride)


CACHE = {"fmt", "reserved", "ck", "cv", "ks", "vs", "pages", "page", "hk", "dim"}
SEQS = {"table", "cu", "lens", "seqs", "width", "stride"}


def _structs(kw):
    c = {("k" if n == "ck" else "v" if n == "cv" else n): kw.pop(n) for n in list(kw) if n in CACHE}
    s = {n: kw.pop(n) for n in list(kw) if n in SEQS}
    return cache_struct(**c), seqs_struct(**s)


def append(q=A, k=A, v=A, xt=0, q_out=A, pos=None, inv=A, rot=64, layout=0, tokens=3, heads=4, qs=256, kstr=128, vstr=128,
           null=(), **kw):
    c, s = _structs(kw)
    r = kv._Rope(inv, rot, layout, 1.0)
    b = [None if n in null else ctypes.byref(x) for n, x in (("rope", r), ("cache", c), ("seqs", s))]
    return mxq.lib().mxq_kv_append(q, k, v, xt, q_out, pos, *b, tokens, heads, qs, kstr, vstr, None)


def attn(q=A, out=A, lse=None, tokens=3, heads=4, qs=256, scale=1.0, window=0, max_q=1, ws=A, ws_bytes=1 << 40, null=(),
         **kw):
    c, s = _structs(kw)
    b = [None if n in null else ctypes.byref(x) for n, x in (("cache", c), ("seqs", s))]
    return mxq.lib().mxq_paged_attn(q, out, lse, *b, tokens, heads, qs, scale, window, max_q, ws, ws_bytes, None)


def test_rope_refusals():
    assert rope(xt=2) == FORMAT and rope(yt=-1) == FORMAT and rope(layout=2) == FORMAT and rope(layout=-1) == FORMAT
    for a in ("x", "y", "pos", "inv"):
        assert rope(**{a: None}) == NULLPTR, a
    assert rope(null_rope=True) == NULLPTR
    for bad in (0, -1):
        assert rope(tokens=bad) == SHAPE and rope(heads=bad) == SHAPE and rope(dim=bad) == SHAPE
    assert rope(rot=-16) == SHAPE and rope(rot=8) == SHAPE and rope(rot=80) == SHAPE and rope(dim=72, rot=64) == SHAPE
    assert rope(xs=255) == SHAPE and rope(ys=64) == SHAPE
    assert rope(x=A, y=A, xt=0, yt=1) == SHAPE and rope(x=A, y=A, yt=0, ys=512) == SHAPE  # in place: same type and stride
    assert rope(x=A + 8) == ALIGN and rope(y=A + 4) == ALIGN and rope(pos=A + 2) == ALIGN and rope(inv=A + 1) == ALIGN
    assert rope(xs=257) == ALIGN and rope(ys=260) == ALIGN
    assert rope(tokens=1 << 31) == UNSUPPORTED and rope(dim=1040, rot=64, xs=4160, ys=4160) == UNSUPPORTED
    assert rope(xs=1 << 29) == UNSUPPORTED


def test_append_refusals():
    assert append(xt=2) == FORMAT and append(layout=7) == FORMAT and append(fmt=1, ks=A, vs=A) == FORMAT
    assert append(fmt=0, ks=A) == FORMAT and append(reserved=1) == FORMAT
    for a in ("k", "v", "inv", "ck", "cv", "table", "cu", "lens"):
        assert append(**{a: None}) == NULLPTR, a
    for n in ("rope", "cache", "seqs"):
        assert append(null=(n,)) == NULLPTR, n
    assert append(q=None) == NULLPTR and append(q_out=None) == NULLPTR
    assert append(fmt=2, ks=A, vs=None) == NULLPTR and append(fmt=2, ks=None, vs=A) == NULLPTR
    for bad in (0, -1):
        for a in ("tokens", "heads", "pages", "page", "hk", "dim", "seqs", "width"):
            assert append(**{a: bad}) == SHAPE, a
    assert append(heads=3) == SHAPE and append(page=24) == SHAPE and append(stride=2) == SHAPE
    assert append(rot=72) == SHAPE and append(rot=80) == SHAPE and append(qs=255) == SHAPE
    assert append(kstr=127) == SHAPE and append(vstr=0) == SHAPE
    for a in ("q", "k", "v", "q_out", "ck", "cv"):
        assert append(**{a: A + 8}) == ALIGN, a
    for a in ("pos", "inv", "table", "cu", "lens"):
        assert append(**{a: A + 2}) == ALIGN, a
    assert append(fmt=2, ks=A + 4, vs=A) == ALIGN and append(qs=257) == ALIGN and append(kstr=130) == ALIGN
    assert append(tokens=(1 << 22) + 1) == UNSUPPORTED and append(page=8) == UNSUPPORTED and append(page=2048) == UNSUPPORTED
    assert append(dim=96, rot=96, qs=384, kstr=192, vstr=192) == UNSUPPORTED
    assert append(seqs=4097) == UNSUPPORTED and append(width=1 << 27, stride=1 << 27) == UNSUPPORTED
    assert append(pages=1 << 31) == UNSUPPORTED and append(qs=1 << 37) == UNSUPPORTED


def test_attention_refusals():
    assert attn(fmt=3) == FORMAT and attn(fmt=0, vs=A) == FORMAT and attn(reserved=5) == FORMAT
    for a in ("q", "out", "ck", "cv", "table", "cu", "lens"):
        assert attn(**{a: None}) == NULLPTR, a
    for n in ("cache", "seqs"):
        assert attn(null=(n,)) == NULLPTR, n
    for bad in (0, -1):
        for a in ("tokens", "heads", "pages", "page", "hk", "dim", "seqs", "width", "max_q"):
            assert attn(**{a: bad}) == SHAPE, a
    assert attn(window=-1) == SHAPE
    assert attn(scale=math.inf) == SHAPE and attn(scale=math.nan) == SHAPE and attn(scale=-2.0 ** 101) == SHAPE
    assert attn(heads=5) == SHAPE and attn(page=48) == SHAPE and attn(qs=255) == SHAPE and attn(ws_bytes=-1) == SHAPE
    for a in ("q", "out", "ws", "ck", "cv"):
        assert attn(**{a: A + 8}) == ALIGN, a
    assert attn(lse=A + 2) == ALIGN and attn(qs=260) == ALIGN and attn(cu=A + 1) == ALIGN
    assert attn(tokens=(1 << 22) + 1) == UNSUPPORTED and attn(dim=32, qs=128) == UNSUPPORTED
    assert attn(tokens=(1 << 23) // 4 + 1, heads=16, qs=1024) == UNSUPPORTED  # more than 2^25 query rows
    assert attn(seqs=4096, hk=2048, heads=2048, qs=2048 * 64) == UNSUPPORTED
    assert attn(window=1 << 31) == UNSUPPORTED and attn(seqs=5000) == UNSUPPORTED


def test_workspace_is_asked_for():
    c, s = cache_struct(hk=2, dim=128, pages=4096, page=64), seqs_struct(seqs=1, width=4096, stride=4096)
    need = mxq.lib().mxq_paged_attn_workspace(ctypes.byref(c), ctypes.byref(s), 1, 8, 1)
    assert need >= 0
    if need:
        kw = dict(tokens=1, qs=1024, heads=8, pages=4096, page=64, dim=128, seqs=1, width=4096, stride=4096)
        assert attn(ws=None, **kw) == NULLPTR and attn(ws_bytes=need - 1, **kw) == SHAPE
    assert mxq.lib().mxq_paged_attn_workspace(None, ctypes.byref(s), 1, 8, 1) == -1
    assert mxq.lib().mxq_paged_attn_workspace(ctypes.byref(c), ctypes.byref(s), 1, 7, 1) == -1
    assert mxq.lib().mxq_paged_attn_workspace(ctypes.byref(c), ctypes.byref(s), 1, 8, 0) == -1


@pytest.mark.skipif(torch.cuda.device_count() != 0, reason="it would launch on fake pointers")
def test_accepted_calls_reach_the_device_check():
    assert rope() == DEVICE and rope(rot=0, inv=None) == DEVICE and rope(x=A, y=A, xt=1, yt=1) == DEVICE
    assert append() == DEVICE and append(q=None, q_out=None) == DEVICE and append(fmt=2, ks=A, vs=A + 8) == DEVICE
    assert append(rot=0, inv=None, page=1024) == DEVICE and append(tokens=1 << 22, seqs=4096) == DEVICE
    assert attn() == DEVICE and attn(lse=A, window=5, max_q=1 << 40) == DEVICE and attn(fmt=2, ks=A, vs=A) == DEVICE


def test_binding_rejects():
    cpu = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        mxq.KVCache(cpu, cpu)
    with pytest.raises(TypeError):
        mxq.rope(torch.zeros(1, 1, 16), torch.zeros(1, dtype=torch.int32), torch.zeros(8))
    with pytest.raises(ValueError):
        mxq.kv_cache(1, 1, 16, 64, fmt="fp16")
    with pytest.raises(ValueError):
        mxq.rope_inv_freq(64, scaling="other")
    with pytest.raises(mxq.MxqError):
        mxq.rope_inv_freq(63)


def test_inverse_frequencies():
    """Each scaling from its definition in Python floats; the table is rounded once."""
    n, theta = 64, 10000.0
    base = [theta ** (-2 * i / n) for i in range(n // 2)]

    def same(got, want):
        assert all(abs(g - w) <= 2.0 ** -24 * w * 1.001 for g, w in zip(got.tolist(), want))

    f, m = mxq.rope_inv_freq(n, theta, device="cpu")
    same(f, base)
    assert m == 1.0
    same(mxq.rope_inv_freq(n, theta, "linear", factor=4, device="cpu")[0], [b / 4 for b in base])
    t2 = theta * 8 ** (n / (n - 2))
    f, m = mxq.rope_inv_freq(n, theta, "ntk", factor=8, device="cpu")
    same(f, [t2 ** (-2 * i / n) for i in range(n // 2)])
    assert abs(f[-1].item() * 8 / base[-1] - 1) < 1e-6 and m == 1.0  # the slowest frequency is divided by the factor
    f, m = mxq.rope_inv_freq(n, theta, "yarn", factor=16, context=4096, low=1, high=32, device="cpu")
    first = math.floor(n / 2 * math.log(4096 / (32 * 2 * math.pi)) / math.log(theta))
    last = math.ceil(n / 2 * math.log(4096 / (1 * 2 * math.pi)) / math.log(theta))
    ramp = [min(1, max(0, (i - first) / (last - first))) for i in range(n // 2)]
    same(f, [b * (1 - r) + b / 16 * r for b, r in zip(base, ramp)])
    assert abs(m - (0.1 * math.log(16) + 1)) < 1e-6 and f[0] == 1.0
    f, m = mxq.rope_inv_freq(n, theta, "bands", factor=8, context=8192, low=1, high=4, device="cpu")
    keep = [min(1, max(0, (8192 * b / (2 * math.pi) - 1) / 3)) for b in base]
    same(f, [k * b + (1 - k) * b / 8 for b, k in zip(base, keep)])
    assert m == 1.0


def test_inverse_frequency_refusals():
    buf = (ctypes.c_float * 512)()
    p, ms = ctypes.addressof(buf), ctypes.c_float()

    def call(sc=0, rot=64, theta=1e4, factor=2.0, context=4096.0, low=1.0, high=32.0, inv=p, m=ctypes.addressof(ms)):
        return mxq.lib().mxq_rope_inv_freq(sc, rot, theta, factor, context, low, high, inv, m)
    assert call() == OK and call(sc=4) == OK and call(rot=2) == OK and call(sc=2, rot=2) == OK and call(rot=1024) == OK
    assert call(sc=5) == FORMAT and call(sc=-1) == FORMAT and call(inv=None) == NULLPTR and call(m=None) == NULLPTR
    assert call(rot=0) == SHAPE and call(rot=7) == SHAPE and call(theta=1.0) == SHAPE and call(theta=math.nan) == SHAPE
    assert call(sc=1, factor=0.5) == SHAPE and call(sc=3, context=0.0) == SHAPE and call(sc=3, low=32.0) == SHAPE
    assert call(sc=4, low=0.0) == SHAPE and call(sc=3, high=math.inf) == SHAPE and call(rot=1026) == UNSUPPORTED


def test_sizes_whose_products_pass_64_bits():
    """Refused by their own limit, whatever a product of them would wrap to."""
    assert append(seqs=1 << 62, hk=4, heads=4, kstr=256, vstr=256) == UNSUPPORTED
    assert attn(seqs=1 << 62, hk=4) == UNSUPPORTED
    assert rope(xs=1 << 62) == UNSUPPORTED and append(qs=1 << 62) == UNSUPPORTED and attn(qs=1 << 62) == UNSUPPORTED
    assert rope(xs=(1 << 62) + 1) == ALIGN
    assert rope(heads=1 << 62) == SHAPE and append(heads=1 << 62, hk=1 << 62) == SHAPE
    assert append(width=1 << 62, stride=1 << 62) == UNSUPPORTED and append(page=1 << 62) == UNSUPPORTED
