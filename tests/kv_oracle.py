"""The calls on the 16-bit paged cache in 64 bits, written from their definitions (include/slope_kv.h), and how far fp32
sums and one bf16 rounding of the softmax weights may be off them."""
import math

import torch


class Batch:
    """Sequences over a paged cache whose free places hold NaN: lens[b] tokens of which the last new[b] are queries."""

    def __init__(self, lens, new, Hq, Hkv, dqk, dv, page, *, seed=0, token_major=False, extra_pages=3, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.Hq, self.Hkv, self.dqk, self.dv, self.page = lens, new, Hq, Hkv, dqk, dv, page
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + extra_pages
        order = torch.randperm(self.n_pages, generator=g)
        self.table = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)  # unused entries: no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].int()
            at += n
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)

        def rows(*shape):
            return (torch.randn(shape, generator=g) * size).to(torch.bfloat16)

        self.q = rows(self.cu[-1], Hq, dqk)
        self.keys = [rows(n, Hkv, dqk) for n in lens]
        self.values = [rows(n, Hkv, dv) for n in lens]

        def pool(parts, d):
            shape = (self.n_pages, page, Hkv, d) if token_major else (self.n_pages, Hkv, page, d)
            x = torch.full(shape, math.nan, dtype=torch.bfloat16)
            view = x.transpose(1, 2) if token_major else x
            for b, part in enumerate(parts):
                for t in range(0, part.shape[0], page):
                    rows = part[t:t + page]
                    view[int(self.table[b, t // page]), :, :rows.shape[0]] = rows.transpose(0, 1)
            return x

        self.k, self.v = pool(self.keys, dqk), pool(self.values, dv)
        self.token_major = token_major

    def slot(self, b, t):
        return int(self.table[b, t // self.page]) * self.page + t % self.page


def visible(n, m, window):
    """[m, n]: which of n tokens the last m see."""
    pos = torch.arange(n - m, n)[:, None]
    gap = pos - torch.arange(n)
    return (gap >= 0) & (gap < window) if window else gap >= 0


def attention(batch, *, window=0, scale=0.0, missing=None):
    """(out [T, Hq, dv], lse [Hq, T], how far out may be off before its rounding, how far lse may be).

    missing(b) -> bool [tokens]: tokens whose page does not exist.
    The kernel's scores are fp32 sums of dqk exact products (off by at most 2^-18 of the sum of their sizes: dqk / 2
    roundings at most one after another, 2^-24 each, with room); a weight is off by that, by the exponent's 2^-21 and by its
    rounding to bf16, 2^-8; the sum and the output's fp32 sums by 2^-18 of their parts' sizes.
    """
    T, Hq, group = batch.cu[-1], batch.Hq, batch.Hq // batch.Hkv
    scale = scale if scale > 0 else batch.dqk ** -0.5
    out = torch.zeros(T, Hq, batch.dv, dtype=torch.float64)
    off = torch.zeros_like(out)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64)
    lse_off = torch.zeros_like(lse)
    for b, (n, m) in enumerate(zip(batch.lens, batch.new)):
        if m == 0:
            continue
        at = slice(batch.cu[b], batch.cu[b + 1])
        k = batch.keys[b].double().repeat_interleave(group, 1)
        v = batch.values[b].double().repeat_interleave(group, 1)
        q = batch.q[at].double()
        s = torch.einsum("ihc,jhc->hij", q, k) * scale
        wobble = torch.einsum("ihc,jhc->hij", q.abs(), k.abs()) * scale * 2.0 ** -18
        seen = visible(n, m, window)
        if missing is not None:
            seen = seen & ~missing(b)
        s = s.masked_fill(~seen, -math.inf)
        wobble = wobble.masked_fill(~seen, 0.0)
        if n == 0:
            continue
        x = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(x == -math.inf, 0.0, x)[..., None])
        lse[:, at] = x
        out[at] = torch.einsum("hij,jhc->ihc", p, v)
        worst = wobble.amax(-1) + 2.0 ** -21 * (s.masked_fill(~seen, 0.0).abs().amax(-1) + 1) * 1.5
        spread = torch.einsum("hij,jhc->ihc", p, v.abs())
        off[at] = spread * (2.0 ** -8 + 2 * worst.t()[..., None] + 2.0 ** -17)
        lse_off[:, at] = worst + 2.0 ** -18 + 2.0 ** -22 * torch.where(x == -math.inf, 0.0, x).abs()
    return out, lse, off, lse_off


def token_weights(batch, lse, *, window=0, scale=0.0):
    """For each sequence (w [Hkv, tokens], how far it may be off), of an lse [Hq, T] as it is.

    Per weight the score's error as in attention(), that of the exponent's argument (2^-22 of its parts' sizes in log2
    units, three roundings), the exponential's 2^-21; the sums of up to thousands of rows 2^-17.
    """
    group = batch.Hq // batch.Hkv
    scale = scale if scale > 0 else batch.dqk ** -0.5
    res = []
    for b, (n, m) in enumerate(zip(batch.lens, batch.new)):
        at = slice(batch.cu[b], batch.cu[b + 1])
        k = batch.keys[b].double().repeat_interleave(group, 1)
        q = batch.q[at].double()
        s = torch.einsum("ihc,jhc->hij", q, k) * scale
        wobble = torch.einsum("ihc,jhc->hij", q.abs(), k.abs()) * scale * 2.0 ** -18
        x = lse[:, at].double()[..., None]
        none = x == -math.inf
        p = torch.exp(s - torch.where(none, 0.0, x))
        p = torch.where(visible(n, m, window) & ~none, p, 0.0)
        part = p * (wobble + 2.0 ** -21 * (1 + 1.5 * (s.abs() + torch.where(none, 0.0, x).abs())) + 2.0 ** -17)
        res.append(tuple(y.sum(1).unflatten(0, (batch.Hkv, group)).sum(1) for y in (p, part)))
    return res


def choose(w, keep, first, recent):
    """Positions, in order, of the `keep` tokens that stay of weights w [tokens]."""
    n = w.shape[0]
    if n <= keep:
        return list(range(n))
    w = w.tolist()

    def size(t):
        x = w[t]
        return (0, 0.0) if x != x else (1, x)

    mid = sorted(range(first, n - recent), key=lambda t: (-size(t)[0], -size(t)[1], t))
    return list(range(first)) + sorted(mid[:keep - first - recent]) + list(range(n - recent, n))
