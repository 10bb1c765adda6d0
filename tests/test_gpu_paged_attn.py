"""Attention over a paged cache against its definition in 64 bits.

Tolerance, derived, per output with A = sum p |v| and S = the largest scale *
sum |q k| of its row: rounding the output 2^-8 |o|; rounding the softmax weights
to bf16 (rows of long chunks) 2 * 2^-8 A, or, as a pair of bf16 (few rows) 2 *
2^-16 A; the fp32 scores are off by at most (dim + 8) 2^-24 S each, which moves
numerator and denominator by that factor each; exponentials, sums over the keys
and the joins of partial results (2^-20 A).  A score also passes through the
factor log2 e in fp32, 2 * 2^-24 S more."""
import math

import pytest
import torch

import block_float_quantized_mxq_amd as mxq
from gpu_util import say
from kv_util import DEV, Case

pytestmark = pytest.mark.gpu


def _check(c, what, window=0, scale=None, max_q=None, few_rows=False, poke=None, cache=None, ref=None):
    say(what)
    scale = c.dim ** -0.5 if scale is None else scale
    cache = c.cache() if cache is None else cache
    out = torch.full((c.tokens, c.heads, c.dim), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.tokens, c.heads), 7.0, device=DEV)
    mxq.paged_attn(c.q16.to(DEV), cache, *c.meta(), scale=scale, window=window, max_q=max_q or c.max_q, out=out, lse=lse)
    ref, mag, reach, ref_lse = ref or c.attention(scale, window)
    o, ls = out.cpu().double(), lse.cpu().double()
    own = slice(c.front, c.tokens - c.behind)
    rest = torch.ones(c.tokens, dtype=torch.bool)
    rest[own] = False
    assert (o[rest] == 7).all() and (ls[rest] == 7).all(), f"{what}: rows of no sequence were written"
    score = 2 * (c.dim + 10) * 2.0 ** -24 * reach
    weights = 2.0 ** -15 if few_rows else 2.0 ** -7
    tol = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + mag * (weights + 2.0 ** -20 + score[..., None]) * (1 + 2.0 ** -7) + 1e-38
    o, ref_, tol = o[own], ref[own], tol[own]
    nan = ref_.isnan()
    assert torch.equal(o.isnan(), nan), f"{what}: NaN in {int(o.isnan().sum())} outputs, expected {int(nan.sum())}"
    bad = ~((o - ref_).abs() <= tol) & ~nan
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {bad.nonzero()[0].tolist()}: "
                           f"{o[bad][0]} against {ref_[bad][0]}")
    ls, rl = ls[own], ref_lse[own]
    fine = torch.isfinite(rl)
    assert torch.equal(ls[~fine].isnan(), rl[~fine].isnan()) and torch.equal(ls[~fine] == -math.inf, rl[~fine] == -math.inf)
    assert ((ls - rl).abs()[fine] <= (score[own] + 2.0 ** -20 * (1 + rl.abs()))[fine]).all(), f"{what}: lse"
    return out


HEADS = [(40, 8, 128), (32, 4, 128), (4, 4, 64), (7, 1, 64), (3, 1, 256), (16, 2, 256), (12, 4, 128), (33, 1, 64)]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
def test_decode(heads, kv_heads, dim, fmt):
    for page, lens in ((16, [1, 2, 15, 16, 17, 63, 64, 65, 333]), (128, [127, 128, 129, 1, 700])):
        c = Case([(1, n) for n in lens], heads, kv_heads, dim, fmt, page, seed=heads + page, front=1, behind=2, table_pad=3)
        _check(c, f"decode {heads}/{kv_heads}/{dim} {fmt} page {page}", few_rows=heads // kv_heads <= 16)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
def test_chunks(heads, kv_heads, dim, fmt):
    c = Case([(5, 5), (0, 0), (70, 200), (33, 33), (1, 90), (0, 17), (130, 131)], heads, kv_heads, dim, fmt, 32,
             seed=heads, behind=1)
    _check(c, f"chunks {heads}/{kv_heads}/{dim} {fmt}")


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(5, 1, 128, 16), (4, 2, 64, 64)])
def test_windows(heads, kv_heads, dim, page, window, fmt):
    c = Case([(1, 300), (150, 260), (1, 3), (2, 129)], heads, kv_heads, dim, fmt, page, seed=window)
    _check(c, f"window {window} {heads}/{kv_heads}/{dim} {fmt}", window=window)
    d = Case([(1, 300), (1, 64), (1, 65)], heads, kv_heads, dim, fmt, page, seed=window + 1)
    _check(d, f"window {window} decode {fmt}", window=window, few_rows=True)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
def test_page_sizes(page, fmt):
    c = Case([(1, 513), (40, 100), (3, 7)], 10, 2, 128, fmt, page, seed=page)
    _check(c, f"page {page} {fmt}")
    _check(Case([(1, 1025), (1, 16), (2, 90)], 10, 2, 128, fmt, page, seed=page), f"page {page} {fmt} decode", few_rows=True)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("new", [1, 2, 3, 4, 8, 16, 31])
def test_few_tokens_over_a_long_context(new, fmt):
    """Long contexts are split over workgroups and joined."""
    c = Case([(new, 4099)], 8, 2, 128, fmt, 64, seed=new)
    _check(c, f"{new} tokens over 4099 {fmt}", few_rows=new * 4 <= 16)


def test_hint_does_not_change_what_is_right():
    c = Case([(3, 200), (45, 45), (1, 500)], 8, 2, 64, "bf16", 16, seed=3)
    ref = c.attention(0.125)
    for hint in (1, 2, 45, 1000000):
        _check(c, f"max_q {hint}", max_q=hint, ref=ref)


@pytest.mark.parametrize("few", [False, True])
def test_rows_that_see_nothing(few):
    """kv_lens below the number of new tokens: rows before position 0 are empty (zeros, lse -inf)."""
    c = Case([(9, 4), (3, 0), (2, 2)] if not few else [(3, 1), (2, 0), (1, 1)], 4, 2, 128, "bf16", 16, seed=4)
    out = _check(c, f"empty rows {few}", few_rows=False)
    assert not out[:2].any()


@pytest.mark.parametrize("new", [2, 5, 60, 200])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_masked_rows_that_are_not_finite(new, fmt, bad):
    """A key or value that is NaN or infinite reaches only the tokens that see it."""
    c = Case([(new, new + 50), (1, 40)], 6, 2, 64, fmt, 16, seed=new)
    p = new + 50 - 1 - new // 3  # seen by the last new // 3 + 1 tokens
    at, r = int(c.table[0, p // 16]), p % 16
    for name, c0 in (("v", 0), ("k", 1)):
        x, sc = c.half[name]
        if fmt == "bf16":
            x[at, c0, r, 3] = float(bad)
            if bad == "inf" and name == "k":
                x[at, c0, r, 3] = float("nan")  # an infinite key: scores of either sign, not a NaN pattern
        else:
            sc[at, c0, r] = 255
    scale = 0.125
    ref = c.attention(scale)
    if bad == "inf" and fmt == "bf16":
        # 64-bit sums give the infinity itself: compare its sign, then take it out of the comparison
        out = torch.empty(c.tokens, c.heads, c.dim, dtype=torch.bfloat16, device=DEV)
        mxq.paged_attn(c.q16.to(DEV), c.cache(), *c.meta(), scale=scale, max_q=c.max_q, out=out)
        inf = ref[0].isinf()
        assert inf.any() and torch.equal(out.cpu().double()[inf], ref[0][inf])
        fine = ref[0].isfinite()
        assert torch.equal(out.cpu().isfinite(), fine)
        assert ((out.cpu().double() - ref[0]).abs()[fine] <= 2.0 ** -6 * ref[1][fine]).all()
    else:
        _check(c, f"masked {bad} {new} {fmt}", scale=scale, ref=ref)


def test_pages_out_of_range_give_nan_to_who_sees_them():
    for seqs, few in (([(1, 100), (1, 40)], True), ([(80, 100), (30, 40)], False)):
        c = Case(seqs, 4, 2, 128, "bf16", 16, seed=8)
        for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
            c.table[0, 3] = bad  # positions 48 .. 63
            _check(c, f"page {bad}", few_rows=few)


def test_lengths_beyond_the_table_and_strange_metadata():
    """Lengths past the table, sequences whose rows pass the tokens: nothing outside is read or written."""
    c = Case([(2, 60), (1, 30)], 4, 2, 128, "bf16", 16, seed=21)
    table, cu, lens = c.meta()
    lens2 = lens.clone()
    lens2[0] = 2 ** 31 - 1
    out = mxq.paged_attn(c.q16.to(DEV), c.cache(), table, cu, lens2)
    assert out.shape == c.q16.shape
    cu2 = torch.tensor([0, 2 ** 30, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    mxq.paged_attn(c.q16.to(DEV), c.cache(), table, cu2, lens)
    cu3 = torch.tensor([5, 3, -9], dtype=torch.int32, device=DEV)
    mxq.paged_attn(c.q16.to(DEV), c.cache(), table, cu3, lens)
    q, k, v = c.qkv()
    for cc in (cu2, cu3):
        mxq.kv_append(k, v, c.cache(), table, cc, lens2, q=q)
    torch.cuda.synchronize()


def test_sharp_and_flat_softmax():
    """Scores of hundreds (one key takes all) and none (the mean)."""
    c = Case([(1, 300), (70, 200)], 8, 2, 128, "bf16", 32, seed=17, q_gain=60.0)
    _check(c, "sharp")
    c.q16.zero_()
    _check(c, "flat")


def test_many_sequences():
    """More sequences than a wave has lanes, some without new tokens."""
    seqs = [((i * 7) % 3, (i * 13) % 50 + 3) for i in range(200)]
    c = Case(seqs, 4, 1, 64, "bf16", 16, seed=19, front=3, behind=5)
    _check(c, "200 sequences")


def test_determinism_streams_and_graphs():
    """The same bits on every run, on another stream, and from a replayed graph whose lengths grow."""
    c = Case([(1, 700), (1, 90), (1, 333)], 40, 8, 128, "mxfp8", 16, seed=23)
    cache, (table, cu, lens), q = c.cache(), c.meta(), c.q16.to(DEV)
    first = mxq.paged_attn(q, cache, table, cu, lens, max_q=1)
    for _ in range(3):
        assert torch.equal(mxq.paged_attn(q, cache, table, cu, lens, max_q=1), first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = mxq.paged_attn(q, cache, table, cu, lens, max_q=1, stream=side)
    side.synchronize()
    assert torch.equal(other, first)
    out = torch.empty_like(first)
    ws = torch.empty(max(1, mxq.paged_attn_workspace(cache, table, cu, lens, 3, 40, 1)), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.paged_attn(q, cache, table, cu, lens, max_q=1, out=out, workspace=ws)
    for step in range(4):
        lens.sub_(step)  # other lengths, same graph
        out.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mxq.paged_attn(q, cache, table, cu, lens, max_q=1))


def test_two_graphs_share_a_workspace():
    cases = [Case([(1, 900)], 8, 2, 128, "bf16", 16, seed=29), Case([(2, 700), (1, 60)], 8, 2, 128, "bf16", 16, seed=30)]
    sides = []
    size = 1
    for c in cases:
        sides.append((c.cache(), *c.meta(), c.q16.to(DEV)))
        size = max(size, mxq.paged_attn_workspace(*sides[-1][:4], c.tokens, 8, c.max_q))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    graphs = []
    for c, (cache, table, cu, lens, q) in zip(cases, sides):
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mxq.paged_attn(q, cache, table, cu, lens, max_q=c.max_q, out=out, workspace=ws)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), c, (cache, table, cu, lens, q) in zip(graphs, cases, sides):
            out.zero_()
            g.replay()
        for (g, out), c, (cache, table, cu, lens, q) in zip(graphs, cases, sides):
            assert torch.equal(out, mxq.paged_attn(q, cache, table, cu, lens, max_q=c.max_q))


def test_a_decode_layer_from_projection_to_projection():
    """The operators as they are used: quantized QKV projection, append with rotation, attention, quantized output
    projection, for a prompt and then three single tokens; the reference recomputes it from what each step stored."""
    hidden, h, hk, d, page = 512, 8, 2, 64, 16
    g = torch.Generator().manual_seed(31)

    def weight(n, k):
        return mxq.quantize(mxq.MXFP4, (torch.randn(n, k, generator=g) * k ** -0.5).bfloat16().to(DEV))

    wqkv, wo = weight((h + 2 * hk) * d, hidden), weight(hidden, h * d)
    dense = {n: mxq.dequant(mxq.MXFP4, *w).double().cpu() for n, w in (("qkv", wqkv), ("o", wo))}
    for fmt in ("bf16", "mxfp8"):
        cache = mxq.kv_cache(8, hk, page, d, fmt)
        table = torch.tensor([[5, 0, 3, 7]], dtype=torch.int32, device=DEV)
        inv, _ = mxq.rope_inv_freq(d, device=DEV)
        held = 0
        for new in (21, 1, 1, 1):
            x = torch.randn(new, hidden, generator=g).bfloat16().to(DEV)
            rows = (mxq.gemm(mxq.MXFP4, *wqkv, x, out_dtype=torch.float32) if new > 8
                    else mxq.gemv(mxq.MXFP4, *wqkv, x))
            q, k, v = (t.unflatten(1, (-1, d)) for t in rows.split([h * d, hk * d, hk * d], 1))
            held += new
            cu = torch.tensor([0, new], dtype=torch.int32, device=DEV)
            lens = torch.tensor([held], dtype=torch.int32, device=DEV)
            q16 = mxq.kv_append(k, v, cache, table, cu, lens, q=q, inv_freq=inv)
            o = mxq.paged_attn(q16, cache, table, cu, lens, max_q=new)
            flat = o.reshape(new, h * d)
            y = mxq.gemm(mxq.MXFP4, *wo, flat, out_dtype=torch.float32) if new > 8 else mxq.gemv(mxq.MXFP4, *wo, flat)
            # the projection in 64 bits: the kernel's own bound
            ref_rows = x.cpu().double() @ dense["qkv"].t()
            bound = 1e-5 * (x.cpu().double().abs() @ dense["qkv"].abs().t()) + 1e-6
            assert ((rows.cpu().double() - ref_rows).abs() <= bound).all()
            ref_y = flat.cpu().double() @ dense["o"].t()
            bound = 1e-5 * (flat.cpu().double().abs() @ dense["o"].abs().t()) + 1e-6
            assert ((y.cpu().double() - ref_y).abs() <= bound).all()
            # the attention over what the cache holds
            c = Case([(new, held)], h, hk, d, fmt, page, seed=1)
            c.table, c.width, c.pages, c.q16 = table.cpu(), 4, 8, q16.cpu()
            c.half = {"k": (cache.k.cpu(), None if fmt == "bf16" else cache.k_scales.cpu()),
                      "v": (cache.v.cpu(), None if fmt == "bf16" else cache.v_scales.cpu())}
            ref, mag, _, _ = c.attention(d ** -0.5)
            assert ((o.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -6.9 * mag).all()


def test_offsets_past_4_gib():
    pages, page, hk, d = 1100, 1024, 16, 128
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v = (torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for t in (k, v):
        t[-2:] = torch.randn(2, hk, page, d, generator=g, device=DEV).bfloat16()
    cache = mxq.KVCache(k, v)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    for new in (1, 40):
        q = torch.randn(new, hk, d, generator=g, device=DEV).bfloat16()
        out = mxq.paged_attn(q, cache, table, torch.tensor([0, new], dtype=torch.int32, device=DEV),
                             torch.tensor([1500], dtype=torch.int32, device=DEV), max_q=new)
        kk = torch.cat([k[-1], k[-2]], 1)[:, :1500].double()
        vv = torch.cat([v[-1], v[-2]], 1)[:, :1500].double()
        a = (q.double().transpose(0, 1) @ kk.transpose(1, 2).contiguous()) * d ** -0.5
        a = a.masked_fill(torch.arange(1500, device=DEV)[None] > torch.arange(1500 - new, 1500, device=DEV)[:, None], -math.inf)
        w = torch.softmax(a, -1)
        ref, mag = (w @ vv).transpose(0, 1), (w @ vv.abs()).transpose(0, 1)
        assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -6.9 * mag).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(24, 24, 64, 16), (48, 24, 128, 32), (24, 24, 256, 16)])
def test_tiles_of_many_rows(heads, kv_heads, dim, page, fmt):
    """Many heads, so that even short chunks go to tiles of 128 rows: odd lengths, a window, empty rows, sequences
    of few rows beside them."""
    for seqs, window in (([(17, 17), (33, 64), (64, 65), (1, 77)], 0), ([(40, 25), (20, 0), (18, 18), (0, 0)], 0),
                         ([(50, 150), (2, 90)], 37)):
        _check(Case(seqs, heads, kv_heads, dim, fmt, page, seed=dim + window, front=1, behind=1),
               f"many rows {seqs} {window}", window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tiles_of_many_rows_with_missing_pages_and_values_that_are_not_finite(dim):
    c = Case([(80, 100), (30, 40)], 24, 24, dim, "bf16", 16, seed=dim)
    for p, h, e in ((75, 1, dim - 2), (90, 23, 3), (99, 7, 40)):
        c.half["v"][0][int(c.table[0, p // 16]), h, p % 16, e] = float("nan")
    c.half["k"][0][int(c.table[1, 1]), 5, 9, 17] = float("nan")
    _check(c, f"not finite {dim}")
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        c.table[0, 3] = bad  # positions 48 .. 63
        _check(c, f"page {bad} {dim}")
    c = Case([(60, 110), (1, 40)], 48, 24, dim, "mxfp8", 16, seed=dim + 1)
    c.half["v"][1][int(c.table[0, 80 // 16]), 3, 80 % 16] = 255
    c.half["k"][1][int(c.table[0, 95 // 16]), 9, 95 % 16, 0] = 255
    _check(c, f"not finite mxfp8 {dim}")


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 64), (8, 1, 128), (16, 2, 256)])
def test_few_tiles_of_few_rows(heads, kv_heads, dim, fmt):
    """Up to 32 tiles of 16 rows: the same result whichever kernel takes them, and just beyond."""
    for seqs in ([(3, 700)], [(13, 1900)], [(32, 400)], [(64, 90), (1, 9)], [(70, 1030)]):
        _check(Case(seqs, heads, kv_heads, dim, fmt, 64, seed=len(seqs) + dim), f"few tiles {seqs}")


@pytest.mark.parametrize("fmt_dim", [64, 128, 256])
@pytest.mark.parametrize("new,heads,kv_heads", [(1, 8, 2), (30, 4, 1), (40, 24, 24)])
def test_an_infinite_value_makes_its_element_infinite(new, heads, kv_heads, fmt_dim):
    """Wherever it lies: among keys that every row sees (a weight as two bf16 would make NaN of it), in another share,
    at the end."""
    c = Case([(new, 1500)], heads, kv_heads, fmt_dim, "bf16", 16, seed=new)
    for p, e, sign in ((5, 3, 1), (700, 9, -1), (1200, 20, 1), (1500 - new, 31, -1), (1499, 40, 1)):
        c.half["v"][0][int(c.table[0, p // 16]), 0, p % 16, e] = sign * math.inf
    scale = c.dim ** -0.5
    out = mxq.paged_attn(c.q16.to(DEV), c.cache(), *c.meta(), scale=scale, max_q=new).cpu().double()
    ref, mag = c.attention(scale)[:2]
    fine = ref.isfinite()
    assert (~fine).sum() >= 4 * new and torch.equal(out[~fine], ref[~fine]) and torch.equal(out.isfinite(), fine)
    assert ((out - ref).abs()[fine] <= 2.0 ** -6 * mag[fine]).all()
