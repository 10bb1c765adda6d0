"""Cases of a paged cache and the definitions of rope, kv_append and paged_attn in
64 bits on the CPU (torch, one sequence and one head at a time)."""
from __future__ import annotations

import math

import torch

import block_float_quantized_mxq_amd as mxq

DEV = "cuda:0"
NAN_BF16, NAN_E4M3 = 0x7FC0, 0x7F


def mx8(v):
    """fp32 [..., d] -> E4M3 codes, E8M0 scales (the MX conversion; finite input)."""
    b = v.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp(-127, 127)
    p = torch.ldexp(b.double(), -e.double()).clamp(-448.0, 448.0).float()
    return p.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)


def mx8_values(codes, scales):
    v = codes.contiguous().view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
    unit = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return (v * unit[..., None]).flatten(-2)


class Case:
    """seqs: (new tokens, cached positions with them) pairs.  Every cache row that no sequence holds, and every unused
    table entry, is poisoned: NaN rows, page ids out of range."""

    def __init__(self, seqs, heads, kv_heads, dim, fmt, page, seed=0, front=0, behind=0, table_pad=0, x="fp32",
                 q_gain=2.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.heads, self.kv_heads, self.dim, self.fmt, self.page = seqs, heads, kv_heads, dim, fmt, page
        self.front, self.behind = front, behind
        need = [-(-max(n, 0) // page) for _, n in seqs]
        width = max(need + [1])
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((len(seqs), width + table_pad), -7, dtype=torch.int32)
        table[:, ::2] = pages + 5
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
        self.width, self.pages = width, pages
        self.table = table
        new = [a for a, _ in seqs]
        self.cu = torch.tensor([front] + new).cumsum(0).to(torch.int32)
        self.lens = torch.tensor([n for _, n in seqs], dtype=torch.int32)
        self.tokens = front + sum(new) + behind
        shape = (pages, kv_heads, page, dim)
        held = torch.zeros(pages, page, dtype=torch.bool)
        for s, (_, n) in enumerate(seqs):
            for p in range(need[s]):
                held[table[s, p], :min(page, n - p * page)] = True
        self.held = held[:, None, :].expand(pages, kv_heads, page)
        self.half = {}
        for name in ("k", "v"):
            v = torch.randn(shape, generator=g).bfloat16()
            if fmt == "bf16":
                v.view(torch.int16)[~self.held] = NAN_BF16
                self.half[name] = (v, None)
            else:
                codes, scales = mx8(v)
                codes[~self.held] = NAN_E4M3
                scales[~self.held] = 255
                self.half[name] = (codes, scales)
        row = torch.randn(self.tokens, (heads + 2 * kv_heads) * dim, generator=g)
        self.row = row if x == "fp32" else row.bfloat16()
        self.q16 = (q_gain * row[:, :heads * dim]).bfloat16().unflatten(1, (heads, dim))

    # device side
    def cache(self):
        (k, ks), (v, vs) = self.half["k"], self.half["v"]
        return mxq.KVCache(*(None if t is None else t.to(DEV) for t in (k, v, ks, vs)))

    def meta(self):
        return self.table.to(DEV)[:, :self.width], self.cu.to(DEV), self.lens.to(DEV)

    def qkv(self):
        h, hk, d = self.heads, self.kv_heads, self.dim
        return [t.unflatten(1, (-1, d)) for t in self.row.to(DEV).split([h * d, hk * d, hk * d], 1)]

    @property
    def max_q(self):
        return max(1, max(a for a, _ in self.seqs))

    # definitions
    def cached(self, name, s, c):
        """Rows of sequence s, key/value head c, in 64 bits; a page out of range: NaN."""
        n = max(0, min(int(self.lens[s]), self.width * self.page))
        x, sc = self.half[name]
        out = torch.full((n, self.dim), float("nan"), dtype=torch.float64)
        for p in range(-(-n // self.page)):
            at, rows = int(self.table[s, p]), min(self.page, n - p * self.page)
            if 0 <= at < self.pages:
                v = x[at, c, :rows]
                out[p * self.page:p * self.page + rows] = v.double() if sc is None else mx8_values(v, sc[at, c, :rows])
        return out

    def attention(self, scale, window=0):
        """(out, sum p |v|, largest scale * sum |q k| of a row, lse) in 64 bits; rows of no sequence: NaN."""
        h, hk, d = self.heads, self.kv_heads, self.dim
        g = h // hk
        nan = float("nan")
        out = torch.full((self.tokens, h, d), nan, dtype=torch.float64)
        mag, reach, lse = out.clone(), torch.full((self.tokens, h), nan, dtype=torch.float64), None
        lse = reach.clone()
        for s, (new, n) in enumerate(self.seqs):
            t0 = int(self.cu[s])
            for c in range(hk):
                k, v = self.cached("k", s, c), self.cached("v", s, c)
                for i in range(new):
                    p = n - new + i
                    hi = min(max(0, p + 1), k.shape[0])
                    lo = max(0, p - window + 1) if window else 0
                    q = self.q16[t0 + i, c * g:(c + 1) * g].double()
                    sl = slice(c * g, (c + 1) * g)
                    if hi <= lo:
                        out[t0 + i, sl], mag[t0 + i, sl], reach[t0 + i, sl], lse[t0 + i, sl] = 0, 0, 0, -math.inf
                        continue
                    kk, vv = k[lo:hi], v[lo:hi]
                    a = scale * (q @ kk.t())
                    w = torch.softmax(a, -1)
                    out[t0 + i, sl] = w @ vv
                    mag[t0 + i, sl] = w @ vv.abs()
                    reach[t0 + i, sl] = scale * (q.abs() @ kk.abs().t()).amax(-1)
                    lse[t0 + i, sl] = torch.logsumexp(a, -1)
        return out, mag, reach, lse


def attention_on(c, device, scale, window=0):
    """Case.attention with one masked product per sequence and key/value head, in 64 bits on the device."""
    g = c.heads // c.kv_heads
    out = torch.full((c.tokens, c.heads, c.dim), float("nan"), dtype=torch.float64, device=device)
    mag, lse = out.clone(), out[..., 0].clone()
    reach = lse.clone()
    for s, (new, n) in enumerate(c.seqs):
        if new == 0:
            continue
        t0 = int(c.cu[s])
        p = torch.arange(n - new, n, device=device)[:, None]
        for h in range(c.kv_heads):
            k, v = c.cached("k", s, h).to(device), c.cached("v", s, h).to(device)
            j = torch.arange(k.shape[0], device=device)[None]
            seen = (j <= p) & (j > p - window if window else j >= 0)
            for i in range(g):
                q = c.q16[t0:t0 + new, h * g + i].to(device).double()
                a = scale * (q @ k.t().contiguous())
                a = torch.where(seen, a, -math.inf)
                w = torch.softmax(a, -1)
                # what a row does not see does not reach it, whatever it is
                bad_v = ~v.isfinite().all(-1)
                sl = (slice(t0, t0 + new), h * g + i)
                clean = torch.where(bad_v[:, None], 0.0, v)
                out[sl], mag[sl] = w @ clean, w @ clean.abs()
                hit = (seen & bad_v[None]).any(-1)
                out[sl] = torch.where(hit[:, None], float("nan"), out[sl])
                kc = torch.nan_to_num(k, 0.0, 0.0, 0.0)
                r = scale * torch.where(seen, q.abs() @ kc.abs().t().contiguous(), 0.0).amax(-1)
                reach[sl], lse[sl] = r, torch.logsumexp(a, -1)
    return tuple(t.cpu() for t in (out, mag, reach, lse))


def turned(x, pos, inv_freq, layout, mscale):
    """(rotation of x [t, h, d] in 64 bits, |a| + |b| of each element's pair)."""
    x = x.double()
    out, mag = x.clone(), torch.zeros_like(x)
    n = inv_freq.numel()
    w = pos.double()[:, None] * inv_freq.double()[None]
    c, s = torch.cos(w)[:, None], torch.sin(w)[:, None]
    i, j = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = mscale * (a * c - b * s), mscale * (b * c + a * s)
    mag[..., i] = mag[..., j] = mscale * (a.abs() + b.abs())
    return out, mag
