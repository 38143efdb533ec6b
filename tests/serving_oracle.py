"""Plain forms of the serving calls in 64 bits (torch on the CPU), from the formulas in include/slope_serving.h.

They share no code with the library: the cache's layout is stated here by the address of every code.
"""
import math

import torch

GROUP, BLOCK = 32, 16
FIFTEENTH = torch.tensor(1.0 / 15.0, dtype=torch.float32)


# ---------------------------------------------------------------- norm and rotation

def norm_rope(x, weight, eps, pos, inv_freq, begin, interleaved, factor, norm=True):
    """(result, size of the pair each channel belongs to), fp64."""
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    out, size = y.clone(), y.abs()
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a = begin + (2 * i if interleaved else i)
        b = begin + (2 * i + 1 if interleaved else half + i)
        t = [math.fmod(p * f, 2 * math.pi) for p in pos.tolist()]
        c = factor * torch.tensor([math.cos(v) for v in t], dtype=torch.float64)[:, None]
        s = factor * torch.tensor([math.sin(v) for v in t], dtype=torch.float64)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = abs(factor) * torch.hypot(y[..., a], y[..., b])
    return out, size


# ---------------------------------------------------------------- the 4-bit cache

def quantise(x):
    """codes, scale, min of x [T, H, d] (bf16 or fp32): [T, H, d] int64, and [T, H, d / 32] bf16 each."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low = g.amin(-1).to(torch.bfloat16)
    span = g.amax(-1) - low.float()
    bad = ~torch.isfinite(g).all(-1) | ~torch.isfinite(low.float()) | ~torch.isfinite(span)
    scale = (span * FIFTEENTH).to(torch.bfloat16)
    zero = bad | ~(scale.float() >= 2.0 ** -126)
    scale = torch.where(zero, torch.zeros_like(scale), scale)
    low = torch.where(bad, torch.full_like(low, math.nan), low)
    step = torch.where(zero, torch.ones_like(scale), scale).double()
    code = ((g.double() - low.double()[..., None]) / step[..., None]).round().clamp(0, 15)
    code = torch.where(zero[..., None], torch.zeros_like(code), code)
    return code.long().flatten(-2), scale, low


def values(code, scale, low):
    """What codes stand for, fp64."""
    return low.double().repeat_interleave(GROUP, -1) + scale.double().repeat_interleave(GROUP, -1) * code.double()


def from_middle(code, scale, low):
    """What the rounding of weight * scale is multiplied by: scale * |code - 8|, and 2^-10 of the scale for the middle's
    own terms, which are fp32 sums of up to 16 scales each (2^-20 of them, over a thousand steps)."""
    return scale.double().repeat_interleave(GROUP, -1) * ((code - 8).abs().double() + 2.0 ** -10)


def block_bytes(dqk, dv):
    return BLOCK * (dqk // 2 + dv // 2 + 4 * (dqk + dv) // GROUP)


def code_address(t, c, d, value, dqk):
    """(byte in the block, high nibble?) of channel c of token t."""
    if value:
        g, code = c % 32 // 4, c % 4 + 4 * (c % 64 // 32)
        at = BLOCK * dqk // 2 + (c // 64 * 32 + 4 * g + t % 8 // 2) * 16 + 4 * (t % 2 + 2 * (t // 8))
    else:
        q, code, w = c % 32 // 8, c % 8, t // 8 * (d // 32) + c // 32
        at = (w // 4 * 32 + 4 * (t % 8) + q) * 16 + 4 * (w % 4)
    return at + code // 2, code % 2


def write_bytes(data, slots, k, v, page_size):
    """Writes into cache bytes data [pages, H, page_size / 16, block] (uint8, CPU), token by token."""
    dqk, dv = k.shape[2], v.shape[2]
    ngk, words = dqk // GROUP, (dqk + dv) // GROUP
    parts = [(x, False) for x in (quantise(k),)] + [(x, True) for x in (quantise(v),)]
    for row, slot in enumerate(slots.tolist()):
        if slot < 0 or slot >= data.shape[0] * page_size:
            continue
        block = data[slot // page_size, :, slot % page_size // BLOCK]
        t = slot % BLOCK
        for (code, scale, low), value in parts:
            d = code.shape[2]
            for c in range(d):
                at, high = code_address(t, c, d, value, dqk)
                n = code[row, :, c].to(torch.uint8)
                old = block[:, at]
                block[:, at] = (old & 0x0F) | (n << 4) if high else (old & 0xF0) | n
            for G in range(d // GROUP):
                at = BLOCK * (dqk + dv) // 2 + 4 * (t * words + (ngk if value else 0) + G)
                word = torch.empty((low.shape[1], 2), dtype=torch.bfloat16)
                word[:, 0], word[:, 1] = low[row, :, G], scale[row, :, G]
                block[:, at:at + 4] = word.view(torch.uint8)


# ---------------------------------------------------------------- attention over known values

def decode(q, k, v, spread, kv_len, q_len, window, scale):
    """One sequence: q [q_len, Hq, dqk], k [keys, H, dqk], v [keys, H, dv], spread = from_middle of the values (fp64).

    Returns out, lse and, for the bounds, sum p * spread, sum p * |v| per output, and the largest
    sum of |q| |k| of a row's visible scores."""
    Hq, H = q.shape[1], k.shape[1]
    out = torch.zeros((q_len, Hq, v.shape[2]), dtype=torch.float64)
    lse = torch.full((Hq, q_len), -math.inf, dtype=torch.float64)
    wide, size = torch.zeros_like(out), torch.zeros_like(out)
    reach = torch.zeros((Hq, q_len), dtype=torch.float64)
    for i in range(q_len):
        pos = kv_len - q_len + i
        lo = max(0, pos - window + 1) if window else 0
        if pos < lo:
            continue
        for h in range(Hq):
            g = h // (Hq // H)
            x = (k[lo:pos + 1, g] @ q[i, h].double()) * scale
            lse[h, i] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[h, i])
            out[i, h] = p @ v[lo:pos + 1, g]
            wide[i, h] = p @ spread[lo:pos + 1, g]
            size[i, h] = p @ v[lo:pos + 1, g].abs()
            reach[h, i] = (k[lo:pos + 1, g].abs() @ q[i, h].double().abs()).max() * scale
    return out, lse, wide, size, reach
