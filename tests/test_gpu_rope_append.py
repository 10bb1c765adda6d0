"""Rotary positions and the paged append against their definitions in 64 bits.

Tolerances, derived: an angle is reduced in double and rounded once to fp32 (at
most pi/4 * 2^-24), sine and cosine are within 2 ulp (2^-22), the rotation adds
three fp32 roundings (2^-24 each, mscale's included); all relative to |a| + |b|
of the pair: together below 2^-21.  A bf16 output adds half a step, 2^-8 |y|.
An E4M3 output adds 2^-4 |y|, or half its smallest step 2^-10 times the block's
scale, and saturates at 448 scales where a block's largest value reaches 512."""
import pytest
import torch

import block_float_quantized_mxq_amd as mxq
from gpu_util import say
from kv_util import DEV, Case, mx8, mx8_values, turned

pytestmark = pytest.mark.gpu
FP32_REL, BF16_REL = 2.0 ** -21, 2.0 ** -8


def _assert_turned(y, ref, mag, bf16, what):
    y = y.detach().cpu().double()
    tol = FP32_REL * mag + (BF16_REL * (ref.abs() + FP32_REL * mag) if bf16 else 0) + 1e-38
    bad = ~((y - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("xt,yt", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 16, 16), (3, 5, 128, 128), (17, 40, 128, 64), (2, 3, 64, 0),
                                                  (9, 2, 256, 32), (1, 56, 128, 128), (65, 1, 1024, 1024),
                                                  (5, 7, 80, 48)])
def test_rope(tokens, heads, dim, rot, xt, yt, layout):
    say("rope", tokens, heads, dim, rot, xt, yt, layout)
    g = torch.Generator().manual_seed(tokens * 131 + dim + rot)
    wide = torch.randn(tokens, heads * dim + 32, generator=g)
    wide = wide if xt == "fp32" else wide.bfloat16()
    pos = torch.randint(0, 200000, (tokens,), generator=g, dtype=torch.int32)
    inv, mscale = (mxq.rope_inv_freq(rot, 10000.0, "yarn", factor=8, context=4096, device="cpu") if rot
                   else (torch.empty(0), 1.0))
    x = wide.to(DEV)[:, 16:16 + heads * dim].unflatten(1, (heads, dim))  # a slice of a wider row
    before = x.clone()
    odt = torch.float32 if yt == "fp32" else torch.bfloat16
    y = mxq.rope(x, pos.to(DEV), inv.to(DEV), layout=layout, mscale=mscale, out_dtype=odt)
    assert torch.equal(x, before) and y.dtype == odt
    ref, mag = turned(wide[:, 16:16 + heads * dim].unflatten(1, (heads, dim)), pos, inv, layout, mscale)
    _assert_turned(y, ref, mag, yt == "bf16", "rope")
    rest = y[..., rot:]
    assert torch.equal(rest, before[..., rot:].to(odt))  # beyond the rotated part: the input, rounded at most


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_far_positions_and_theirs_signs(layout):
    """Positions over the whole int32 range turn as exactly as small ones."""
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    inv, _ = mxq.rope_inv_freq(64, 500000.0, device="cpu")
    x = torch.randn(pos.numel(), 3, 64, generator=torch.Generator().manual_seed(5))
    y = mxq.rope(x.to(DEV), pos.to(DEV), inv.to(DEV), layout=layout, out_dtype=torch.float32)
    ref, mag = turned(x, pos, inv, layout, 1.0)
    # the definition's own angle in double is off by 2^-53 of up to 2^31: 2.4e-7
    assert ((y.cpu().double() - ref).abs() <= (FP32_REL + 2.4e-7) * mag + 1e-38).all()
    assert torch.equal(y[0].cpu(), x[0])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope_in_place_equals_out_of_place(layout, dtype):
    x = torch.randn(33, 6 * 128, generator=torch.Generator().manual_seed(6)).to(DEV).to(dtype)
    pos = torch.arange(33, dtype=torch.int32, device=DEV) * 997
    inv, _ = mxq.rope_inv_freq(96, device=DEV)
    view = x[:, 128:640].unflatten(1, (4, 128))
    want = mxq.rope(view, pos, inv, layout=layout, out_dtype=dtype)
    untouched = x[:, :128].clone(), x[:, 640:].clone()
    got = mxq.rope(view, pos, inv, layout=layout, out=view)
    assert got.data_ptr() == view.data_ptr() and torch.equal(view, want)
    assert torch.equal(x[:, :128], untouched[0]) and torch.equal(x[:, 640:], untouched[1])


def _positions(c):
    pos = torch.zeros(c.tokens, dtype=torch.int64)
    for s, (new, n) in enumerate(c.seqs):
        pos[int(c.cu[s]):int(c.cu[s]) + new] = torch.arange(n - new, n)
    return pos


SEQS = {
    "one token": [(1, 1)],
    "decode": [(1, 1), (1, 16), (1, 17), (1, 333)],
    "chunks with empty sequences": [(0, 0), (5, 5), (0, 40), (33, 70), (0, 0), (1, 2), (0, 9)],
    "pages end inside": [(50, 83), (31, 31), (64, 64)],
}


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("xt", ["fp32", "bf16"])
@pytest.mark.parametrize("name,heads,kv_heads,dim,page,rot,layout", [
    ("one token", 40, 8, 128, 16, 128, "half"), ("decode", 32, 4, 128, 64, 64, "interleaved"),
    ("chunks with empty sequences", 6, 2, 64, 16, 64, "half"), ("pages end inside", 3, 1, 256, 32, 32, "half"),
    ("chunks with empty sequences", 8, 8, 128, 1024, 128, "interleaved"), ("pages end inside", 4, 4, 64, 16, 0, "half")])
def test_append(name, heads, kv_heads, dim, page, rot, layout, xt, fmt):
    say("append", name, heads, kv_heads, dim, page, rot, layout, xt, fmt)
    c = Case(SEQS[name], heads, kv_heads, dim, fmt, page, seed=dim + rot, front=2, behind=3, table_pad=3, x=xt)
    cache = c.cache()
    old = [None if t is None else t.cpu().clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    q, k, v = c.qkv()
    inv = mxq.rope_inv_freq(rot, device="cpu")[0] if rot else None
    q_out = torch.full((c.tokens, heads, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    got = mxq.kv_append(k, v, cache, *c.meta(), q=q, inv_freq=None if inv is None else inv.to(DEV), layout=layout,
                        q_out=q_out)
    assert got is q_out
    pos, inv = _positions(c), torch.empty(0) if inv is None else inv
    own = slice(c.front, c.tokens - c.behind)
    ref, mag = turned(q.cpu(), pos, inv, layout, 1.0)
    _assert_turned(q_out[own], ref[own], mag[own], True, "q_out")
    assert (q_out[:c.front] == 7).all() and (q_out[c.tokens - c.behind:] == 7).all()
    new = {"k": turned(k.cpu(), pos, inv, layout, 1.0), "v": (v.cpu().double(), torch.zeros(v.shape, dtype=torch.float64))}
    for i, part in enumerate(("k", "v")):
        stored = (cache.k, cache.v)[i].cpu()
        scales = (cache.k_scales, cache.v_scales)[i]
        touched = torch.zeros(c.pages, page, dtype=torch.bool)
        for s, (count, n) in enumerate(c.seqs):
            for j in range(count):
                p, t = n - count + j, int(c.cu[s]) + j
                at, r = int(c.table[s, p // page]), p % page
                touched[at, r] = True
                want, pair = new[part][0][t], new[part][1][t]
                if fmt == "bf16":
                    _assert_turned(stored[at, :, r], want, pair, True, f"{part} row {t}")
                else:
                    sc = scales.cpu()[at, :, r]
                    val = mx8_values(stored[at, :, r], sc)
                    unit = torch.exp2(sc.double() - 127).repeat_interleave(32, -1)
                    amax = want.abs().unflatten(-1, (-1, 32)).amax(-1)
                    lo = torch.floor(torch.log2(amax * (1 - 2.0 ** -20))) - 8 + 127
                    hi = torch.floor(torch.log2(amax * (1 + 2.0 ** -20))) - 8 + 127
                    assert ((sc.double() == lo) | (sc.double() == hi)).all()
                    err = (val - want).abs()
                    tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * unit) + FP32_REL * pair
                    tol = torch.maximum(tol, (want.abs() - 448 * unit) * (1 + 2.0 ** -20))
                    assert (err <= tol).all(), f"{part} row {t}: {float((err - tol).max())}"
        kept = ~touched[:, None].expand(-1, kv_heads, -1)
        assert torch.equal(stored.view(torch.uint8 if fmt == "mxfp8" else torch.int16)[kept],
                           old[i].view(torch.uint8 if fmt == "mxfp8" else torch.int16)[kept])
        if scales is not None:
            assert torch.equal(scales.cpu()[kept], old[2 + i][kept])


def test_mxfp8_append_equals_quantizer_bit_for_bit():
    """Values (and unrotated keys) from bf16 rows: the library's own quantizer on the same rows."""
    c = Case([(37, 100), (1, 5)], 4, 2, 128, "mxfp8", 32, seed=9, x="bf16")
    cache = c.cache()
    _, k, v = c.qkv()
    k = k.contiguous()
    k[3, 1, 32:64] = 0.0
    k[4, 0, :32] = 448.0 * 2 ** -3
    k[5, 0, 5] = -511.0
    assert mxq.kv_append(k, v, cache, *c.meta()) is None
    for x, codes, scales in ((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales)):
        qc, qs = mxq.quantize(mxq.MXFP8, x.reshape(-1, 128).contiguous())
        qc, qs = qc.view(-1, 2, 128), qs.view(-1, 2, 4)
        for s, (count, n) in enumerate(c.seqs):
            for j in range(count):
                p, t = n - count + j, int(c.cu[s]) + j
                at = int(c.table[s, p // 32]), slice(None), p % 32
                assert torch.equal(codes[at], qc[t]) and torch.equal(scales[at], qs[t])
    # and the library's decode reads the cache
    w = mxq.dequant(mxq.MXFP8, cache.v.view(-1, 128), cache.v_scales.view(-1, 4)).cpu().double().view(cache.shape)
    vals = mx8_values(cache.v.cpu(), cache.v_scales.cpu())
    assert torch.equal(w[c.held], vals[c.held])


def test_mxfp8_append_marks_blocks_that_are_not_finite():
    c = Case([(4, 4)], 2, 1, 64, "mxfp8", 16, seed=11)
    cache = c.cache()
    _, k, v = c.qkv()
    v = v.contiguous()
    v[1, 0, 3], v[2, 0, 40], v[3, 0, 0] = float("nan"), float("inf"), 3e38
    mxq.kv_append(k, v, cache, *c.meta())
    sc = cache.v_scales.cpu()[int(c.table[0, 0]), 0, :4]
    assert sc[1, 0] == 255 and sc[2, 1] == 255 and sc[2, 0] != 255 and sc[1, 1] != 255 and sc[3, 0] == 127 + 127 - 8


def test_explicit_positions_and_plain_k_equal_rope():
    """bf16 cache rows are bit for bit what rope gives at the same positions."""
    c = Case([(9, 40), (3, 3)], 4, 2, 128, "bf16", 16, seed=12)
    cache = c.cache()
    q, k, v = c.qkv()
    pos = torch.randint(0, 100000, (c.tokens,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).to(DEV)
    inv, _ = mxq.rope_inv_freq(128, device=DEV)
    q_out = mxq.kv_append(k, v, cache, *c.meta(), q=q, inv_freq=inv, positions=pos, mscale=1.25)
    assert torch.equal(q_out, mxq.rope(q, pos, inv, mscale=1.25))
    want = mxq.rope(k, pos, inv, mscale=1.25)
    for s, (count, n) in enumerate(c.seqs):
        for j in range(count):
            p, t = n - count + j, int(c.cu[s]) + j
            assert torch.equal(cache.k[int(c.table[s, p // 16]), :, p % 16], want[t])


def test_tokens_without_a_place_store_nothing():
    """Pages out of range, positions before 0 or beyond the table: queries turn, nothing is stored."""
    c = Case([(4, 2), (3, 40), (2, 20)], 2, 1, 64, "bf16", 16, seed=13)
    table, cu, lens = c.meta()
    table = table.clone()
    table[1, 2] = c.pages  # positions 32 .. 39 of sequence 1
    table[2, 1] = -1       # positions 16 .. 19 of sequence 2
    table = table[:, :3]
    cache = c.cache()
    before = cache.k.view(torch.int16).clone()
    q, k, v = c.qkv()
    inv, _ = mxq.rope_inv_freq(64, device=DEV)
    q_out = mxq.kv_append(k, v, cache, table, cu, lens, q=q, inv_freq=inv)
    changed = (cache.k.view(torch.int16) != before).any(-1).any(1).cpu()
    want = torch.zeros_like(changed)
    want[int(c.table[0, 0]), :2] = True  # tokens 2 and 3 of sequence 0 are positions 0 and 1
    assert torch.equal(changed, want)
    pos = torch.tensor([-2, -1, 0, 1, 37, 38, 39, 18, 19])
    ref, mag = turned(q.cpu(), pos, inv.cpu(), "half", 1.0)
    _assert_turned(q_out, ref, mag, True, "q_out")


def test_large_page_offsets():
    """Rows whose byte offset passes 2^32."""
    pages, page, hk, d = 1100, 1024, 16, 128  # 2 x 4.6 GB
    cache = mxq.KVCache(*(torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    cache.k[-1].zero_(), cache.v[-1].zero_()
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    k = torch.randn(3, hk, d, device=DEV).bfloat16()
    v = torch.randn(3, hk, d, device=DEV).bfloat16()
    mxq.kv_append(k, v, cache, table, torch.tensor([0, 3], dtype=torch.int32, device=DEV),
                  torch.tensor([page], dtype=torch.int32, device=DEV))
    assert torch.equal(cache.k[-1, :, -3:], k.transpose(0, 1)) and torch.equal(cache.v[-1, :, -3:], v.transpose(0, 1))
    assert not cache.k[-1, :, :-3].any()
