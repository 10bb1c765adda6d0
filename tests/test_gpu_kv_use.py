"""The cache operators at the sizes that long prompts run at (8-wave workgroups, split and joined chunks), and as
a server uses them: captured steps, several streams, unusual scales, refusals of the binding.  Tolerances as in the
attention tests."""
import math

import pytest
import torch

import block_float_quantized_mxq_amd as mxq
from gpu_util import say
from kv_util import DEV, Case, attention_on, mx8_values

pytestmark = pytest.mark.gpu


def _run(c, scale, window=0, max_q=None):
    out = torch.full((c.tokens, c.heads, c.dim), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(c.tokens, c.heads, device=DEV)
    mxq.paged_attn(c.q16.to(DEV), c.cache(), *c.meta(), scale=scale, window=window, max_q=max_q or c.max_q, out=out, lse=lse)
    return out.cpu().double(), lse.cpu().double()


def _check(c, what, window=0, scale=None):
    say(what)
    scale = c.dim ** -0.5 if scale is None else scale
    o, lse = _run(c, scale, window)
    ref, mag, reach, ref_lse = attention_on(c, DEV, scale, window)
    score = 2 * (c.dim + 10) * 2.0 ** -24 * reach.abs()
    tol = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + mag * (2.0 ** -7 + 2.0 ** -20 + score[..., None]) * (1 + 2.0 ** -7) + 1e-38
    nan = ref.isnan()
    # (a value that is not finite makes its own element NaN or infinite, the reference the whole row)
    assert (o.isfinite() | nan).all() and not (nan.all(-1) & o.isfinite().all(-1)).any(), what
    bad = ~((o - ref).abs() <= tol) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[0].tolist()}"
    fine = ref_lse.isfinite()
    assert ((lse - ref_lse).abs()[fine] <= (score + 2.0 ** -20 * (1 + ref_lse.abs()))[fine]).all(), f"{what}: lse"


def test_the_large_reference_is_the_definition():
    c = Case([(3, 20), (0, 0), (9, 9), (4, 2)], 6, 2, 64, "mxfp8", 16, seed=2, front=1, behind=1)
    for window in (0, 5):
        a, b = c.attention(0.2, window), attention_on(c, "cpu", 0.2, window)
        for x, y in zip(a[:1], b[:1]):
            seen = a[3].isfinite()
            assert torch.allclose(x[seen], y[seen], rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("seqs,heads,kv_heads,page,window", [
    ([(2100, 2300)], 16, 16, 64, 0), ([(1500, 1501), (777, 900)], 16, 16, 16, 0), ([(2100, 2100)], 16, 16, 32, 100),
    ([(601, 601), (1, 2000), (500, 777)], 40, 8, 128, 0)])
def test_long_prompts(seqs, heads, kv_heads, page, window, fmt):
    """More tiles of 128 rows than compute units: workgroups of 8 waves and 256 rows."""
    _check(Case(seqs, heads, kv_heads, 128, fmt, page, seed=len(seqs) + window), f"long {seqs} {fmt}", window)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("new,total,heads,kv_heads,dim,window", [
    (512, 6000, 40, 8, 128, 0), (130, 9001, 8, 2, 64, 0), (64, 5003, 8, 1, 256, 0), (300, 8192, 32, 4, 128, 2500),
    (33, 3333, 4, 4, 128, 0)])
def test_chunks_over_long_contexts(new, total, heads, kv_heads, dim, window, fmt):
    """Shares of the positions, joined; both workgroup sizes."""
    _check(Case([(new, total)], heads, kv_heads, dim, fmt, 64, seed=new), f"{new} over {total} {dim} {fmt}", window)


def test_long_prompt_with_values_that_are_not_finite_and_missing_pages():
    c = Case([(2100, 2200)], 16, 16, 128, "bf16", 64, seed=40)
    for p in (150, 1031, 2199):
        c.half["v"][0][int(c.table[0, p // 64]), 3, p % 64, 5] = float("nan")
    c.half["k"][0][int(c.table[0, 1500 // 64]), 7, 1500 % 64, 9] = float("nan")
    _check(c, "not finite")
    c.table[0, 20] = -1
    c.table[0, 21] = c.pages
    _check(c, "missing pages")


def test_ragged_batches():
    """Many sequences of every length: decode shares of equal length, tiles whole and split, and a chunk among them."""
    lens = [1 + (i * 7919) % 5000 for i in range(70)]
    _check(Case([(1, n) for n in lens], 8, 2, 128, "bf16", 32, seed=50), "70 ragged")
    _check(Case([(1, 900)] * 40, 16, 8, 64, "mxfp8", 32, seed=51), "40 alike")
    _check(Case([(1, n) for n in lens[:20]] + [(150, 1700)] + [(2, n + 1) for n in lens[20:30]], 8, 2, 128, "mxfp8", 32,
                seed=52), "mixed")


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-30, 3.0])
def test_scales(scale):
    """No scale, a negative one (the softmax prefers the smallest scores), a tiny and a large one."""
    for seqs in ([(1, 200), (2, 70)], [(70, 150)]):
        _check(Case(seqs, 8, 2, 64, "bf16", 16, seed=61, q_gain=1.0), f"scale {scale}", scale=scale)


def test_smallest_block_scales():
    """Scale bytes 0 .. 4: values of up to 448 * 2^-123, the smallest below bf16's normal range.  The decode rounds
    each to bf16's subnormal steps (half of 2^-133, and so their mean), the output to bf16: half a step, 2^-8 of a
    normal value or half of 2^-133."""
    c = Case([(1, 64)], 2, 1, 64, "mxfp8", 64, seed=62, q_gain=0.0)
    codes, scales = c.half["v"]
    scales[int(c.table[0, 0])] = torch.arange(64)[None, :, None].remainder(5).to(torch.uint8)
    o, _ = _run(c, 0.125)
    ref = mx8_values(codes, scales)[int(c.table[0, 0]), 0].mean(0)
    assert ((o[0] - ref[None]).abs() <= 2.0 ** -8 * ref.abs()[None] + 2.0 ** -133).all() and o.abs().max() > 2.0 ** -125


def test_captured_decode_steps():
    """Append and attention of a decode step in one graph: positions come from the lengths on the device, so the graph
    is replayed as they grow, with the program's own work between."""
    h, hk, d, page, n = 8, 2, 128, 16, 3
    for fmt in ("bf16", "mxfp8"):
        g = torch.Generator(device=DEV).manual_seed(70)
        caches = [mxq.kv_cache(40, hk, page, d, fmt) for _ in range(2)]
        table = torch.arange(39, dtype=torch.int32, device=DEV).view(3, 13)
        cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
        lens = torch.tensor([1, 15, 100], dtype=torch.int32, device=DEV)
        row = torch.empty(n, (h + 2 * hk) * d, device=DEV)
        inv, _ = mxq.rope_inv_freq(d, device=DEV)

        def step(cache, out=None):
            q, k, v = (t.unflatten(1, (-1, d)) for t in row.split([h * d, hk * d, hk * d], 1))
            q16 = mxq.kv_append(k, v, cache, table, cu, lens, q=q, inv_freq=inv)
            return mxq.paged_attn(q16, cache, table, cu, lens, max_q=1, out=out)

        row.normal_(generator=g)
        out = torch.empty(n, h, d, dtype=torch.bfloat16, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(caches[0], out)
        for _ in range(12):
            row.normal_(generator=g)
            out.zero_()
            graph.replay()
            want = step(caches[1])
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert torch.equal(caches[0].k.view(torch.uint8), caches[1].k.view(torch.uint8))
            lens += 1


def test_two_streams_at_once():
    """Calls that overlap, each with the workspace that the binding makes for it."""
    cases = [Case([(1, 4000), (1, 70)], 16, 2, 128, "bf16", 16, seed=80), Case([(40, 3000)], 16, 2, 128, "mxfp8", 16, seed=81)]
    held = [(c.q16.to(DEV), c.cache(), *c.meta()) for c in cases]
    want = [mxq.paged_attn(*a, max_q=c.max_q) for a, c in zip(held, cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for a, c, s in zip(held, cases, streams):
            got.append(mxq.paged_attn(*a, max_q=c.max_q, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


def test_binding_refusals():
    c = Case([(2, 40)], 4, 2, 64, "bf16", 16, seed=90)
    cache, (table, cu, lens), q = c.cache(), c.meta(), c.q16.to(DEV)
    for name in ("k", "v", "k_scales", "v_scales"):
        with pytest.raises(AttributeError):
            setattr(cache, name, cache.k)
    with pytest.raises(TypeError):
        mxq.paged_attn(q.float(), cache, table, cu, lens)
    with pytest.raises(TypeError):
        mxq.paged_attn(q, cache, table.long(), cu, lens)
    with pytest.raises(ValueError):
        mxq.paged_attn(q, cache, table, cu[:-1], lens)
    with pytest.raises(ValueError):
        mxq.paged_attn(q[..., :32], cache, table, cu, lens)
    with pytest.raises(ValueError):
        mxq.paged_attn(q.transpose(0, 1), cache, table, cu, lens, out=torch.empty_like(q))
    with pytest.raises(ValueError):
        mxq.paged_attn(q, cache, table, cu, lens, lse=torch.empty(2, 2, device=DEV))
    with pytest.raises(ValueError):
        mxq.paged_attn_workspace(cache, table, cu, lens, 2, 5, 1)
    with pytest.raises(mxq.MxqError):
        mxq.paged_attn(q[:0], cache, table, cu, lens)
    with pytest.raises(mxq.MxqError):
        mxq.paged_attn(q, cache, table, cu, lens, window=-3)
    with pytest.raises(ValueError):
        mxq.KVCache(cache.k, cache.v[:, :, :8].contiguous())
    with pytest.raises(TypeError):
        mxq.KVCache(cache.k, cache.v, cache.k, cache.v)
    row, k, v = c.qkv()
    with pytest.raises(TypeError):
        mxq.kv_append(k, v.bfloat16(), cache, table, cu, lens)
    with pytest.raises(ValueError):
        mxq.kv_append(k, v, cache, table, cu, lens, q_out=q)
    with pytest.raises(ValueError):
        mxq.kv_append(k, v, cache, table, cu, lens, positions=lens)
    with pytest.raises(ValueError):
        mxq.kv_append(k, v, cache, table, cu, lens, layout="other")
    with pytest.raises(ValueError):
        mxq.rope(row, lens, torch.empty(16, device=DEV))
    with pytest.raises(mxq.MxqError):
        mxq.rope(row, cu[:2], torch.empty(12, device=DEV))  # 24 elements: not whole units of 16
    far = torch.empty(64 * 16 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(1, 16, 64)
    with pytest.raises(mxq.MxqError):
        mxq.rope(far, lens, torch.empty(32, device=DEV))  # 2 bytes off the 16-byte alignment


def test_log_sum_exp_joins_two_caches():
    """The use of lse: attention over a prefix and over the rest, joined, is attention over both."""
    c = Case([(1, 300)], 8, 2, 128, "bf16", 16, seed=95)
    q, cache, (table, cu, lens) = c.q16.to(DEV), c.cache(), c.meta()
    whole_lse = torch.empty(1, 8, device=DEV)
    whole = mxq.paged_attn(q, cache, table, cu, lens, lse=whole_lse).double()
    parts = []
    for t, n in ((table[:, :10], 160), (table[:, 10:], 140)):
        lse = torch.empty(1, 8, device=DEV)
        o = mxq.paged_attn(q, cache, t, cu, torch.tensor([n], dtype=torch.int32, device=DEV), lse=lse)
        parts.append((o.double(), lse.double()))
    w = torch.softmax(torch.stack([p[1] for p in parts]), 0)
    joined = sum(wi[..., None] * p[0] for wi, p in zip(w, parts))
    bound = 2.0 ** -8 * (whole.abs() + sum(wi[..., None] * p[0].abs() for wi, p in zip(w, parts))) + 2.0 ** -14
    assert ((joined - whole).abs() <= bound).all()
    total = torch.logsumexp(torch.stack([p[1] for p in parts]), 0)
    assert ((total - whole_lse.double()).abs() <= 2.0 ** -18 * (1 + total.abs())).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("seqs,heads,kv_heads,dim,window", [
    ([(1300, 1500), (3, 400), (40, 90)], 8, 1, 256, 0), ([(900, 900), (700, 2000)], 4, 2, 256, 333),
    ([(210, 700)], 20, 4, 256, 0), ([(1300, 1500), (3, 400), (40, 90)], 6, 2, 64, 0), ([(1800, 1800)], 16, 16, 64, 257)])
def test_long_prompts_of_other_heads(seqs, heads, kv_heads, dim, window, fmt):
    """Heads of 256 (two waves share their rows) and of 64, whole and in shares, with sequences of few rows among them."""
    _check(Case(seqs, heads, kv_heads, dim, fmt, 32, seed=dim + window), f"prompt {dim} {seqs} {fmt}", window)


def test_wide_heads_with_values_that_are_not_finite_and_missing_pages():
    """As for heads of 128: in either half of the elements, and in a prompt that is split."""
    for seqs, heads in (([(700, 820)], 8), ([(60, 2000), (2, 300)], 4)):
        c = Case(seqs, heads, 2, 256, "bf16", 16, seed=70)
        total = seqs[0][1]
        for p, h, e in ((total - 1, 1, 200), (total - 30, 0, 5), (total - 55, 1, 131)):
            c.half["v"][0][int(c.table[0, p // 16]), h, p % 16, e] = float("nan")
        _check(c, f"values {seqs}")
        p = total - 40
        c.half["k"][0][int(c.table[0, p // 16]), 1, p % 16, 250] = float("nan")
        _check(c, f"keys {seqs}")
        c.table[0, (total - 20) // 16] = c.pages
        _check(c, f"pages {seqs}")


def test_rope_refuses_an_output_that_is_no_tensor():
    x = torch.zeros(2, 2, 64, device=DEV)
    pos, inv = torch.zeros(2, dtype=torch.int32, device=DEV), mxq.rope_inv_freq(64)[0]
    for out in ([1], torch.zeros(2, 2, 64), torch.zeros(2, 2, 64, dtype=torch.float16, device=DEV)):
        with pytest.raises(TypeError):
            mxq.rope(x, pos, inv, out=out)


@pytest.mark.parametrize("seqs,heads,kv_heads", [([(1, 300), (2, 90)], 8, 2), ([(60, 200), (1, 90)], 24, 24)])
def test_queries_that_are_slices_of_a_row(seqs, heads, kv_heads):
    """The same bits as from contiguous queries: bf16 slices of a fused row, as a model without rotation has them."""
    c = Case(seqs, heads, kv_heads, 128, "bf16", 16, seed=91)
    q, args = c.q16.to(DEV), (c.cache(), *c.meta())
    row = torch.full((c.tokens, (heads + 2 * kv_heads) * 128 + 8), 9.0, dtype=torch.bfloat16, device=DEV)
    part = row[:, 8:8 + heads * 128].unflatten(1, (heads, 128))
    part.copy_(q)
    assert not part.is_contiguous()
    assert torch.equal(mxq.paged_attn(part, *args, max_q=c.max_q), mxq.paged_attn(q, *args, max_q=c.max_q))


@pytest.mark.parametrize("seqs,heads,kv_heads,dim", [
    ([(200, 900), (1, 700), (2, 60)], 24, 8, 128), ([(40, 3000)], 64, 8, 256), ([(3, 800), (1, 90)], 8, 1, 64)])
def test_captured_chunks(seqs, heads, kv_heads, dim):
    """Chunks beside decode, chunks in shares, and few tiles, captured: replays follow the lengths and the tables."""
    c = Case(seqs, heads, kv_heads, dim, "bf16", 16, seed=92)
    q, cache, (table, cu, lens) = c.q16.to(DEV), c.cache(), c.meta()
    for t in (cache.k, cache.v):
        t.nan_to_num_(nan=0.5)  # rows of no sequence become visible below
    out, lse = torch.empty_like(q), torch.empty(c.tokens, heads, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.paged_attn(q, cache, table, cu, lens, max_q=c.max_q, out=out, lse=lse)
    for _ in range(4):
        out.zero_()
        lse.zero_()
        graph.replay()
        want_lse = torch.empty_like(lse)
        want = mxq.paged_attn(q, cache, table, cu, lens, max_q=c.max_q, lse=want_lse)
        torch.cuda.synchronize()
        # bits: a rolled table has pages that do not exist, and NaN in the rows that see them
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
        lens.sub_(17)
        table.copy_(table.roll(1, 1))


def test_captured_rope():
    x = torch.randn(9, 4, 128, device=DEV)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    inv, _ = mxq.rope_inv_freq(128)
    out = torch.empty(9, 4, 128, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.rope(x, pos, inv, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, mxq.rope(x, pos, inv))
        pos += 1000
        x.normal_()


@pytest.mark.parametrize("new", [1, 3])
def test_the_most_sequences(new):
    """4096 sequences: one key each that is theirs alone, all others share a page."""
    n, h, hk, d = 4096, 8, 2, 64
    g = torch.Generator(device=DEV).manual_seed(93)
    k, v = (torch.randn(n + 1, hk, 16, d, device=DEV, generator=g).bfloat16() for _ in range(2))
    table = torch.stack([torch.full((n,), n, device=DEV), torch.arange(n, device=DEV)], 1).int()
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV) * new
    lens = torch.full((n,), 16 + new, dtype=torch.int32, device=DEV)
    q = torch.randn(n * new, h, d, device=DEV, generator=g).bfloat16()
    out = mxq.paged_attn(q, mxq.KVCache(k, v), table, cu, lens, scale=0.125, max_q=new).double()
    for t in (0, new - 1, 5 * new, 4095 * new, n * new - 1, 2048 * new + new - 1):
        s, i = t // new, t % new
        keys, vals = (torch.cat([x[n], x[s, :, :i + 1]], 1).double() for x in (k, v))
        for head in range(h):
            p = torch.softmax(0.125 * (keys[head // 4] @ q[t, head].double()), 0)
            ref, mag = p @ vals[head // 4], p @ vals[head // 4].abs()
            assert ((out[t, head] - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -12 * mag).all(), (t, head)


def test_a_prompt_of_many_tokens():
    """20000 tokens, sampled: the first, the last, and around the edges of tiles."""
    n, h, hk, d, page = 20000, 16, 2, 128, 64
    g = torch.Generator(device=DEV).manual_seed(94)
    pages = -(-n // page)
    k, v = (torch.randn(pages, hk, page, d, device=DEV, generator=g).bfloat16() for _ in range(2))
    table = torch.randperm(pages, device=DEV, generator=g).int()[None]
    cu, lens = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, n], [n]))
    q = torch.randn(n, h, d, device=DEV, generator=g).bfloat16()
    out = mxq.paged_attn(q, mxq.KVCache(k, v), table, cu, lens)
    flat = [x[table[0].long()].transpose(0, 1).reshape(hk, -1, d) for x in (k, v)]
    for t in (0, 1, 15, 16, 63, 64, 4095, 9999, 19967, 19968, 19999):
        for head in (0, 7, 8, 15):
            keys, vals = (x[head // 8, :t + 1].double() for x in flat)
            p = torch.softmax(keys @ q[t, head].double() * d ** -0.5, 0)
            ref, mag = p @ vals, p @ vals.abs()
            # half a step of the output, and of each weight in numerator only: 2 * 2^-8 of sum p |v| covers both
            assert ((out[t, head].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7 * mag).all(), (t, head)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("seqs,window", [([(2500, 2500)], 0), ([(1300, 1333), (1000, 2000)], 301), ([(2200, 2100)], 0)])
def test_wide_heads_in_many_tiles(seqs, window, fmt):
    """Heads of 256 in more tiles than compute units: workgroups of 128 rows and 8 waves."""
    _check(Case(seqs, 16, 2, 256, fmt, 64, seed=95 + window), f"many tiles {seqs} {fmt}", window)
