"""The serving calls on the GPU against plain forms in 64 bits (tests/serving_oracle.py).

Tolerances, from the arithmetic:

* A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24.
* norm and rotation: an angle is off by at most 2^-24 of a turn (2^-21.3 radians), and fewer than 16 fp32 roundings
  of at most the pair's size follow: 2^-20 of the pair's size, besides the output's own rounding.
* cache: the codes, scales and minimums are exact; a value is one fp32 rounding, then the output's.
* cache attention: weight * scale is rounded to bf16 once and multiplies code - 8, the rest of a value being added in
  fp32 (2^-8 of sum p * scale * |code - 8|); scores are sums of at most 192
  products in fp32, off by at most 2^-18 of sum |q| |k|, which moves a weight by as much again.
* packed prompts: the bounds that the prefill attention's own tests use.
"""
import math
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import oracle
import ring_attention_slope_gb300 as slope
import serving_oracle as so

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    slope.build()
    slope.load()
    assert slope.device_status() == (0, 0)
    yield
    torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)


def rand(*shape, seed=0, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- norm and rotation

def check_rope(got, x, w, eps, pos, freq, begin, inter, factor, norm=True):
    ref, size = so.norm_rope(x, w, eps, pos, freq, begin, inter, factor, norm)
    got = got.cpu()
    tol = HALF[got.dtype] * ref.abs() + 2.0 ** -20 * size + 1e-30
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), ((got.double() - ref).abs() / tol).max()


@pytest.mark.parametrize("T,Hq,Hkv,d,begin,dim,inter", [
    (1, 1, 1, 64, 0, 64, False), (3, 8, 1, 64, 0, 64, True), (5, 3, 3, 64, 16, 16, False), (33, 40, 8, 64, 8, 48, False),
    (7, 5, 1, 128, 0, 128, False), (6, 4, 2, 128, 40, 32, True), (9, 7, 7, 192, 128, 64, True),
    (4, 2, 1, 192, 0, 192, False), (2, 3, 1, 192, 24, 112, False), (300, 12, 4, 64, 0, 32, False),
    (1300, 64, 8, 64, 0, 64, False), (5000, 7, 2, 64, 8, 32, False), (4000, 6, 2, 128, 0, 128, True)])
def test_norm_rope(T, Hq, Hkv, d, begin, dim, inter):
    q, k = rand(T, Hq, d, seed=1, scale=3), rand(T, Hkv, d, seed=2, scale=0.02)
    qw, kw = rand(d, seed=3, dtype=torch.float32), rand(Hkv, d, seed=4)
    freq, factor = slope.rope_inv_freq(dim, scaling="yarn", factor=4, original=2048, fast=32, slow=1)
    pos = torch.randint(-100000, 2000000, (T,), generator=torch.Generator().manual_seed(5))
    rope = slope.Rope(freq, begin=begin, interleaved=inter, attention_factor=factor)
    qo, ko = slope.qk_norm_rope(q.cuda(), k.cuda(), q_weight=qw.cuda(), k_weight=kw.cuda(), eps=1e-5, rope=rope,
                                positions=i32(pos))
    check_rope(qo, q, qw, 1e-5, pos, freq, begin, inter, factor)
    check_rope(ko, k, kw, 1e-5, pos, freq, begin, inter, factor)


@pytest.mark.parametrize("tin", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tout", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128, 192])
def test_norm_rope_types(tin, tout, d):
    q, k = rand(19, 3, d, seed=6, dtype=tin), rand(19, 1, d, seed=7, dtype=tin)
    freq, _ = slope.rope_inv_freq(d)
    qo, ko = slope.qk_norm_rope(q.cuda(), k.cuda(), rope=slope.Rope(freq), pos0=77, out_dtype=tout)
    pos = torch.arange(77, 96)
    check_rope(qo, q, None, 1e-6, pos, freq, 0, False, 1.0)
    check_rope(ko, k, None, 1e-6, pos, freq, 0, False, 1.0)


def test_norm_rope_far_positions():
    """Up to the ends of int32, where an fp32 product of position and frequency would be off by many turns."""
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 1, 999_999_937, 16_777_217])
    q = rand(5, 2, 64, seed=8, dtype=torch.float32)
    freq, _ = slope.rope_inv_freq(64, 500000.0)
    for inter in (False, True):
        qo, ko = slope.qk_norm_rope(q.cuda(), rope=slope.Rope(freq, interleaved=inter), positions=i32(pos), norm=False)
        assert ko is None
        # the oracle's own fp64 angle is off by up to 2^31 * 2^-53 radians
        check_rope(qo, q, None, 0, pos, freq, 0, inter, 1.0, norm=False)


@pytest.mark.parametrize("norm,rotate", [(True, False), (False, True), (False, False)])
def test_norm_or_rope_alone(norm, rotate):
    q, k = rand(21, 4, 128, seed=9), rand(21, 2, 128, seed=10)
    freq, _ = slope.rope_inv_freq(64, scaling="linear", factor=2)
    qo, ko = slope.qk_norm_rope(q.cuda(), k.cuda(), norm=norm, rope=slope.Rope(freq, begin=32) if rotate else None)
    pos = torch.arange(21)
    for x, y in ((q, qo), (k, ko)):
        check_rope(y, x, None, 1e-6, pos, freq if rotate else [], 32, False, 1.0, norm=norm)
        if not norm and not rotate:
            assert torch.equal(y.cpu(), x)


def test_norm_rope_in_place_and_strided():
    """Views into one projection's output [T, (Hq + 2 Hkv) d + 8], rotated in place: the rest of it stays."""
    T, Hq, Hkv, d = 5070, 6, 2, 64  # enough that warps go on to further tokens
    buf = rand(T, (Hq + 2 * Hkv) * d + 8, seed=11)
    dev = buf.cuda()
    view = lambda b, h0, n: b[:, h0 * d:(h0 + n) * d].unflatten(1, (n, d))  # noqa: E731
    freq, _ = slope.rope_inv_freq(d)
    q, k = view(dev, 0, Hq), view(dev, Hq, Hkv)
    slope.qk_norm_rope(q, k, rope=slope.Rope(freq), q_out=q, k_out=k, pos0=5)
    pos = torch.arange(5, 5 + T)
    check_rope(q, view(buf, 0, Hq), None, 1e-6, pos, freq, 0, False, 1.0)
    check_rope(k, view(buf, Hq, Hkv), None, 1e-6, pos, freq, 0, False, 1.0)
    assert torch.equal(dev[:, (Hq + Hkv) * d:].cpu(), buf[:, (Hq + Hkv) * d:])


def test_norm_rope_special_values():
    """A row of zeros stays zero (eps), a NaN or an infinity stays in its own head, no tokens is a no-op."""
    q = rand(4, 2, 64, seed=12)
    q[0, 0] = 0
    q[1, 1, 3] = math.nan
    q[2, 0, 40] = math.inf
    freq, _ = slope.rope_inv_freq(64)
    qo = slope.qk_norm_rope(q.cuda(), rope=slope.Rope(freq))[0].cpu()
    assert torch.equal(qo[0, 0], torch.zeros(64, dtype=torch.bfloat16))
    assert torch.isnan(qo[1, 1]).all()
    assert torch.isnan(qo[2, 0, 40]) and not torch.isnan(qo[2, 0, :8]).any()
    ok = [(0, 1), (1, 0), (2, 1), (3, 0), (3, 1)]
    ref, size = so.norm_rope(q, None, 1e-6, torch.arange(4), freq, 0, False, 1.0)
    for t, h in ok:
        assert ((qo[t, h].double() - ref[t, h]).abs() <= 2.0 ** -8 * ref[t, h].abs() + 2.0 ** -20 * size[t, h]).all()
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert slope.qk_norm_rope(e, e[:, :1], rope=slope.Rope(freq))[0].shape == (0, 2, 64)


# ---------------------------------------------------------------- the cache

def fresh(n_pages, page, H, dqk, dv, fill=0xA5):
    data = torch.full((n_pages, H, page // 16, so.block_bytes(dqk, dv)), fill, dtype=torch.uint8, device="cuda")
    return slope.KV4Cache(n_pages, page, H, dqk, dv, data=data)


def hard(T, H, d, seed, dtype):
    """Values that meet the format's edges: constants, ties, off-centre, tiny, huge, zeros and ordinary groups."""
    x = rand(T, H, d, seed=seed, dtype=torch.float32)
    kind = torch.arange(T * H).view(T, H) % 7
    x[kind == 1] = 1.625
    x[kind == 2] = (x[kind == 2] * 4).round() / 2 + 37  # quotients at halves are common
    x[kind == 3] *= 1e-30
    x[kind == 4] *= 1e30
    x[kind == 5] = 0
    return x.to(dtype)


SHAPES = [(1, 1, 64, 64, 16), (17, 2, 64, 64, 16), (40, 3, 128, 128, 32), (33, 2, 192, 128, 64), (20, 1, 128, 64, 16),
          (25, 2, 64, 128, 128), (19, 2, 192, 64, 1024), (130, 8, 64, 64, 64)]


@pytest.mark.parametrize("T,H,dqk,dv,page", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cache_write_bytes_and_read(T, H, dqk, dv, page, dtype):
    """Every byte of the cache, those of untouched slots too, then the values read back."""
    n_pages = -(-T // page) + 2
    k, v = hard(T, H, dqk, 20, dtype), hard(T, H, dv, 21, dtype)
    slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(22))[:T]
    if T > 4:
        slots[1], slots[2], slots[3] = -1, n_pages * page, -(2 ** 31)
    cache = fresh(n_pages, page, H, dqk, dv)
    want = cache.data.cpu().clone()
    so.write_bytes(want, slots, k, v, page)
    slope.kv4_write(cache, k.cuda(), v.cuda(), i32(slots))
    assert torch.equal(cache.data.cpu(), want)
    live = [t for t, s in enumerate(slots.tolist()) if 0 <= s < n_pages * page]
    for out in (torch.bfloat16, torch.float32):
        ko = torch.full((T, H, dqk), 7.0, dtype=out, device="cuda")
        vo = torch.full((T, H, dv), 7.0, dtype=out, device="cuda")
        slope.kv4_read(cache, i32(slots), k_out=ko, v_out=vo)
        for x, y in ((k, ko.cpu()), (v, vo.cpu())):
            ref = so.values(*so.quantise(x))
            half = HALF[out] + (2.0 ** -24 if out == torch.bfloat16 else 0)
            # fp32 products of numbers near 2^-130 lose bits below the smallest subnormal
            assert ((y.double() - ref).abs()[live] <= half * ref.abs()[live] + 2.0 ** -149).all()
            rest = [t for t in range(T) if t not in live]
            assert (y[rest] == 7).all()
            step = so.quantise(x)[1].double().repeat_interleave(32, -1)
            # half a step, and where the top of the range rounds away: 15 * 2^-8 steps more; fp32 inputs add min's rounding
            slack = 2.0 ** -8 * ref.abs() + (2.0 ** -8 * x.double().abs().amax(-1, keepdim=True) if dtype == torch.float32 else 0)
            assert ((x.double() - ref).abs()[live] <= ((0.5 + 15 * 2.0 ** -8) * step + slack)[live] + 1e-37).all()


def test_cache_groups_that_are_not_finite():
    """A NaN or an infinity, or a range that overflows, takes its own 32 channels along and nothing else."""
    T, H, d = 6, 2, 64
    k, v = rand(T, H, d, seed=23, dtype=torch.float32), rand(T, H, d, seed=24, dtype=torch.float32)
    k[0, 1, 5], v[1, 0, 40], k[2, 0, 33], k[2, 0, 34] = math.nan, math.inf, 3e38, -3e38
    v[3, 1, 0] = -math.inf
    cache = fresh(1, 16, H, d, d)
    slope.kv4_write(cache, k.cuda(), v.cuda(), i32(range(T)))
    want = torch.full((1, H, 1, so.block_bytes(d, d)), 0xA5, dtype=torch.uint8)
    so.write_bytes(want, torch.arange(T), k, v, 16)
    assert torch.equal(cache.data.cpu(), want)
    ko, vo = (x.cpu() for x in slope.kv4_read(cache, i32(range(T)), out_dtype=torch.float32))
    nan_k, nan_v = torch.zeros(T, H, d, dtype=bool), torch.zeros(T, H, d, dtype=bool)
    nan_k[0, 1, :32] = nan_k[2, 0, 32:] = nan_v[1, 0, 32:] = nan_v[3, 1, :32] = True
    assert torch.equal(torch.isnan(ko), nan_k) and torch.equal(torch.isnan(vo), nan_v)


def test_cache_strided_inputs_and_repeated_reads():
    T, H, d, page = 37, 4, 64, 32
    both = rand(T, 2, H + 1, d + 8, seed=25).cuda()
    k, v = both[:, 0, 1:, :d], both[:, 1, :H, 8:]
    cache = fresh(3, page, H, d, d)
    slots = torch.arange(T) + 5
    slope.kv4_write(cache, k, v, i32(slots))
    again = torch.cat([slots, slots.flip(0), slots[:3]])
    out = torch.zeros(again.numel(), 2, H, d + 8, dtype=torch.bfloat16, device="cuda")
    ko, vo = slope.kv4_read(cache, i32(again), k_out=out[:, 0, :, :d], v_out=out[:, 1, :, 8:])
    for x, y in ((k, ko), (v, vo)):
        ref = so.values(*so.quantise(x.cpu().contiguous()))
        ref = torch.cat([ref, ref.flip(0), ref[:3]])
        assert ((y.cpu().double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -24) * ref.abs()).all()
    assert (out[:, 0, :, d:] == 0).all() and (out[:, 1, :, :8] == 0).all()


# ---------------------------------------------------------------- attention over the cache

def paged(lens, page, H, dqk, dv, seed, extra=3, scale=1.0, garbage=True):
    """A cache whose every other byte is garbage (NaN words among it), a table, and each sequence's held k, v."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + extra
    cache = fresh(n_pages, page, H, dqk, dv, fill=0xFF if garbage else 0)  # words 0xffffffff: NaN scale, NaN min
    width = max(need + [1]) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=g)
    at, held = 0, []
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]].int()
        at += need[b]
        k, v = rand(n, H, dqk, seed=seed + 10 * b + 1, scale=scale), rand(n, H, dv, seed=seed + 10 * b + 2, scale=scale)
        if n:
            t = torch.arange(n)
            slots = table[b, (t // page).long()].long() * page + t % page
            slope.kv4_write(cache, k.cuda(), v.cuda(), i32(slots))
        kq, vq = so.quantise(k), so.quantise(v)
        kk, vv = so.values(*kq), so.values(*vq)
        held.append((kk, vv, so.from_middle(*vq)))
    return cache, table, held


def check_decode(out, lse, q, held, lens, q_len, window, scale, rows=None):
    B, Hq = len(lens), q.shape[1]
    out, q = out.cpu(), q.cpu()
    for b in range(B) if rows is None else rows:
        k, v, spread = held[b]
        r0 = b * q_len
        ref, rl, wide, size, reach = so.decode(q[r0:r0 + q_len], k, v, spread, lens[b], q_len, window, scale)
        got, gl = out[r0:r0 + q_len].double(), lse[:, r0:r0 + q_len].cpu().double()
        none = torch.isneginf(rl)
        assert torch.equal(torch.isneginf(gl), none), f"sequence {b}: empty rows"
        assert (got[none.t()] == 0).all()
        err = torch.where(none, torch.zeros_like(gl), gl - rl).abs()
        moved = 2.0 ** -18 * reach + 1e-6
        assert (err <= moved + 2.0 ** -22 * torch.where(none, torch.zeros_like(rl), rl).abs()).all(), (b, err.max())
        tol = 2.0 ** -8 * wide + 2 * moved.t()[..., None] * size + HALF[out.dtype] * ref.abs() + 2.0 ** -20 * size + 1e-30
        assert ((got - ref).abs() <= tol).all(), (b, ((got - ref).abs() / tol).max())


def run_decode(lens, q_len, Hq, H, dqk, dv, page, window=0, seed=40, out_dtype=None, scale=0.0, **kw):
    cache, table, held = paged(lens, page, H, dqk, dv, seed)
    q = rand(len(lens) * q_len, Hq, dqk, seed=seed + 5)
    out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32(lens), q_len=q_len, window=window, scale=scale,
                              out_dtype=out_dtype, **kw)
    check_decode(out, lse, q, held, lens, q_len, window, scale or 1 / math.sqrt(dqk))


@pytest.mark.parametrize("lens", [[1], [0], [16], [17], [255], [1, 0, 5], [64, 63, 65, 1], [300, 2, 0, 129, 700]])
def test_decode_lengths(lens):
    run_decode(lens, 1, 8, 1, 64, 64, 16)


@pytest.mark.parametrize("dqk,dv", [(64, 64), (64, 128), (128, 64), (128, 128), (192, 64), (192, 128)])
@pytest.mark.parametrize("Hq,H,q_len", [(2, 2, 1), (8, 2, 1), (8, 1, 2), (15, 3, 1), (24, 2, 1), (5, 1, 7)])
def test_decode_heads_and_sizes(dqk, dv, Hq, H, q_len):
    """Groups of 1 to 12 query heads, one to seven queries: one tile of 8 rows, one of 16, and several."""
    run_decode([3, 130, 41], q_len, Hq, H, dqk, dv, 32)


@pytest.mark.parametrize("page", [16, 32, 64, 1024])
@pytest.mark.parametrize("window,q_len", [(0, 1), (1, 1), (17, 1), (40, 3), (1000, 2), (5, 64)])
def test_decode_pages_and_windows(page, window, q_len):
    run_decode([100, 1, 33, 259], q_len, 4, 2, 64, 64, page, window=window)


def test_decode_long_and_split():
    """Long enough that many CTAs share a pair, beside short ones that share a CTA."""
    run_decode([9000, 3, 77, 0, 2500, 1], 1, 16, 2, 64, 64, 64, out_dtype=torch.float32)
    run_decode([4100, 20], 3, 4, 4, 192, 128, 16)


def test_decode_many_sequences():
    """More sequences than a CTA has threads, so the range search runs in rounds."""
    lens = [(7 * i) % 50 for i in range(300)]
    run_decode(lens, 1, 8, 1, 64, 64, 16, seed=60)


@pytest.mark.parametrize("lens", [[39] * 10, [64] * 70, [200] * 60, [1024] * 24, [2048] * 12, [1500] + [9] * 100,
                                  [3000, 0, 700] * 5, [40] * 400])
@pytest.mark.parametrize("q_len,dqk,dv", [(1, 64, 64), (3, 192, 128)])
def test_decode_cuts(lens, q_len, dqk, dv):
    """One piece to a CTA or several, whole pairs or shared ones: every kind of cut, and every sequence gets its rows."""
    H, Hq, page = 4, 16, 64
    cache, table, held = paged(lens, page, H, dqk, dv, 62)
    q = rand(len(lens) * q_len, Hq, dqk, seed=63)
    out = torch.full((len(lens) * q_len, Hq, dv), float("nan"), dtype=torch.bfloat16, device="cuda")
    _, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32(lens), q_len=q_len, out=out)
    assert torch.isfinite(out).all()
    pick = sorted({0, 1, len(lens) // 2, len(lens) - 1})
    check_decode(out, lse, q, held, lens, q_len, 0, 1 / math.sqrt(dqk), rows=pick)
    single = [slope.kv4_attn(q[b * q_len:(b + 1) * q_len].cuda(), cache, table[b:b + 1].cuda(), i32(lens[b:b + 1]),
                             q_len=q_len, out_dtype=torch.float32)[0] for b in range(0, len(lens), 7)]
    for b, one in zip(range(0, len(lens), 7), single):  # two bf16 roundings of weights, one of the output
        ours = out[b * q_len:(b + 1) * q_len].float()
        spread = held[b][2].abs().max().item() if lens[b] else 0.0
        assert ((ours - one).abs() <= 2.0 ** -8 * one.abs() + 2.0 ** -6 * spread + 1e-6).all(), b


def test_decode_scale_and_large_scores():
    """A scale of its own; scores whose maximum moves often and whose weights underflow."""
    run_decode([500], 1, 8, 1, 64, 64, 16, scale=0.01)
    run_decode([500, 90], 1, 8, 1, 64, 64, 16, scale=3.0, seed=61)


@pytest.mark.parametrize("qs,ks,vs", [(1e-20, 1.0, 1e-8), (1e10, 1e-10, 1e6), (1.0, 1.0, 1e12), (0.0, 1.0, 1.0),
                                      (1e-38, 1.0, 1.0)])
def test_decode_magnitudes(qs, ks, vs):
    """Query rows and cached values far from one: nothing flushes or overflows in the 16-bit operands."""
    lens, page, H, Hq, d = [200, 31], 16, 1, 8, 64
    cache = fresh(16, page, H, d, d)
    table = torch.arange(16, dtype=torch.int32).view(1, 16).repeat(2, 1)
    table[1] = table[1].flip(0)
    held = []
    for b, n in enumerate(lens):
        k, v = rand(n, H, d, seed=70 + b, scale=ks), rand(n, H, d, seed=80 + b, scale=vs)
        t = torch.arange(n)
        slope.kv4_write(cache, k.cuda(), v.cuda(), i32(table[b, (t // page).long()].long() * page + t % page))
        kq, vq = so.quantise(k), so.quantise(v)
        held.append((so.values(*kq), so.values(*vq), so.from_middle(*vq)))
    q = rand(2, Hq, d, seed=90, scale=qs)
    out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32(lens), out_dtype=torch.float32)
    check_decode(out, lse, q, held, lens, 1, 0, 0.125)


def test_decode_bad_pages_and_lengths():
    """A page outside the cache holds no keys, a negative length is none, a long one ends with the table."""
    lens, page = [64, 64, -5, 10 ** 6], 16
    cache, table, held = paged([64, 64, 64, 64], page, 1, 64, 64, 100)
    table = table[:, :4].contiguous()
    table[1, 1], table[1, 3] = 10 ** 6, -7
    q = rand(4, 8, 64, seed=101)
    out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32(lens))
    keep = torch.cat([torch.arange(0, 16), torch.arange(32, 48)])
    some = [held[0], tuple(x[keep] for x in held[1]), held[2], held[3]]
    check_decode(out, lse, q, some, [64, 32, 0, 64], 1, 0, 0.125)


def test_decode_hidden_values_do_not_leak():
    """NaN groups behind a window, after a query's own position and past the end reach no row that does not see them."""
    page, n = 16, 40
    cache, table, held = paged([n], page, 1, 64, 64, 110)
    k, v = rand(n, 1, 64, seed=111), rand(n, 1, 64, seed=112)
    k[3], v[4], v[39] = math.nan, math.inf, math.nan
    t = torch.arange(n)
    slope.kv4_write(cache, k.cuda(), v.cuda(), i32(table[0, (t // page).long()].long() * page + t % page))
    q = rand(2, 8, 64, seed=113)
    out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32([n]), q_len=2, window=30)
    kq, vq = so.quantise(k), so.quantise(v)
    kk, vv = so.values(*kq), so.values(*vq)
    ref, rl, wide, size, reach = so.decode(q[:1], kk, vv, so.from_middle(*vq), n - 1, 1, 30, 0.125)
    assert torch.isfinite(out[0].float()).all() and torch.isnan(out[1].float()).all()
    assert ((out[:1].cpu().double() - ref).abs() <= 2.0 ** -7 * (wide + size)).all()
    assert torch.isfinite(lse).all()
    # and a row that does see a NaN key is NaN
    out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32([n]), q_len=2)
    assert torch.isnan(out.float()).all() and torch.isnan(lse).all()


def test_decode_strides_and_guards():
    """Strided q, out, lse and table; what lies between is not touched; lse may be left out."""
    lens, Hq, d, page = [50, 7, 90], 8, 64, 32
    cache, table, held = paged(lens, page, 2, d, d, 120)
    qbuf = rand(3, Hq + 1, d + 8, seed=121).cuda()
    q = qbuf[:, 1:, 8:]
    wide = torch.full((3, table.shape[1] + 5), 12345, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    for dtype in (torch.bfloat16, torch.float32):
        obuf = torch.full((5, Hq + 2, d + 8), 9.0, dtype=dtype, device="cuda")
        lbuf = torch.full((3, 2 * Hq), 9.0, device="cuda")
        out, lse = obuf[1:4, 1:-1, :d], lbuf[:, ::2].t()
        slope.kv4_attn(q, cache, wide.cuda()[:, :table.shape[1]], i32(lens), out=out, lse=lse)
        check_decode(out, lse, q, held, lens, 1, 0, 0.125)
        out.fill_(9.0)
        lse.fill_(9.0)
        assert (obuf == 9).all() and (lbuf == 9).all()
        slope.kv4_attn(q, cache, wide.cuda()[:, :table.shape[1]], i32(lens), out=out, want_lse=False)
        assert (lbuf == 9).all() and not (out == 9).all()


def test_decode_same_bits_streams_and_graphs():
    """The same bits from every launch, on another stream, and from a captured graph replayed with new lengths."""
    lens, page = [3000, 17, 500], 64
    cache, table, held = paged(lens, page, 2, 64, 64, 130)
    q, tab, n = rand(3, 16, 64, seed=131).cuda(), table.cuda(), i32(lens)
    out, lse = slope.kv4_attn(q, cache, tab, n)
    for _ in range(3):
        o2, l2 = slope.kv4_attn(q, cache, tab, n)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    torch.cuda.synchronize()
    ws = [torch.empty(slope.kv4_attn_workspace_size(3, 16, cache), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(out) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, w, o in zip(streams, ws, outs):
        with torch.cuda.stream(s):
            for _ in range(4):
                slope.kv4_attn(q, cache, tab, n, out=o, workspace=w)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)
    graph = torch.cuda.CUDAGraph()
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.graph(graph):
        slope.kv4_attn(q, cache, tab, n, out=o3, lse=l3, workspace=ws[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    shorter = [64, 17, 2]
    n.copy_(i32(shorter))
    graph.replay()
    torch.cuda.synchronize()
    check_decode(o3, l3, q, [tuple(x[:m] for x in h) for h, m in zip(held, shorter)], shorter, 1, 0, 0.125)


def test_decode_scores_far_below_zero():
    """One key: weight 1, whatever its score.  A query beyond the documented range gives NaN, not a wrong number."""
    cache, table, held = paged([1, 1], 16, 1, 64, 64, 140)
    q = rand(2, 8, 64, seed=141)
    q[1] = -q[0]  # one of the two scores is negative
    for scale in (1e3, 1e6):
        out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32([1, 1]), scale=scale, out_dtype=torch.float32)
        assert torch.isfinite(lse).all()
        for b in range(2):
            _, v, spread = held[b]
            assert ((out[b].cpu().double() - v[0]).abs() <= 2.0 ** -8 * spread[0] + 2.0 ** -20 * v[0].abs()).all()
    q[1, 3, 5] = 2.0 ** 118
    out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32([1, 1]))
    assert torch.isnan(lse[3, 1]) and torch.isfinite(lse[:3]).all() and torch.isfinite(lse[4:]).all()


def test_decode_on_a_stream_of_its_own():
    """What a call allocates for another stream is not handed out while that stream still uses it."""
    lens = [5000, 40, 900]
    cache, table, held = paged(lens, 64, 2, 64, 64, 150)
    q, tab, n = rand(3, 16, 64, seed=151).cuda(), table.cuda(), i32(lens)
    want, want_lse = slope.kv4_attn(q, cache, tab, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    size = slope.kv4_attn_workspace_size(3, 16, cache)
    results = []
    for _ in range(8):
        results.append(slope.kv4_attn(q, cache, tab, n, stream=side))
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0x7F)  # the workspace's size, on the current stream
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(l, want_lse) for o, l in results)


def test_offsets_past_32_bits():
    """Pages, rows and heads that lie more than 2^32 bytes into their tensors."""
    page, H, d = 1024, 8, 64
    n_pages = 2 ** 32 // slope.serving.load().slope_kv4_cache_bytes(1, page, H, d, d) + 40
    cache = slope.KV4Cache(n_pages, page, H, d, d)
    assert cache.data.numel() > 2 ** 32
    n = 1500
    table = torch.tensor([[n_pages - 1, 3], [1, n_pages - 7]], dtype=torch.int32)
    held, t = [], torch.arange(n)
    for b in range(2):
        k, v = rand(n, H, d, seed=160 + b), rand(n, H, d, seed=170 + b)
        slots = i32(table[b, t // page].long() * page + t % page)
        slope.kv4_write(cache, k.cuda(), v.cuda(), slots)
        kq, vq = so.quantise(k), so.quantise(v)
        held.append((so.values(*kq), so.values(*vq), so.from_middle(*vq)))
        ko, vo = slope.kv4_read(cache, slots)
        assert ((ko.cpu().double() - held[b][0]).abs() <= (2.0 ** -8 + 2.0 ** -24) * held[b][0].abs()).all()
        assert ((vo.cpu().double() - held[b][1]).abs() <= (2.0 ** -8 + 2.0 ** -24) * held[b][1].abs()).all()
    q = rand(2, 16, d, seed=180)
    out, lse = slope.kv4_attn(q.cuda(), cache, table.cuda(), i32([n, n]))
    check_decode(out, lse, q, held, [n, n], 1, 0, 0.125)
    del cache
    # rows 2^26 elements apart
    T, Hq, row = 40, 4, 2 ** 26
    buf = torch.empty(T * row, dtype=torch.bfloat16, device="cuda")
    q, k, v = (buf.as_strided((T, h, d), (row, d, 1), at) for h, at in ((Hq, 0), (1, 1024), (1, 2048)))
    xq, xk, xv = rand(T, Hq, d, seed=190), rand(T, 1, d, seed=191), rand(T, 1, d, seed=192)
    for dst, src in ((q, xq), (k, xk), (v, xv)):
        dst.copy_(src.cuda())
    qo, ko = buf.as_strided((T, Hq, d), (row, d, 1), 4096), buf.as_strided((T, 1, d), (row, d, 1), 8192)
    slope.qk_norm_rope(q, k, rope=slope.Rope([0.5] * 32), q_out=qo, k_out=ko)
    for got, x in ((qo, xq), (ko, xk)):
        check_rope(got.contiguous(), x, None, 1e-6, torch.arange(T), [0.5] * 32, 0, False, 1.0)
    out = buf.as_strided((T, Hq, d), (row, d, 1), 16384)
    slope.attn_varlen(q, k, v, [0, 15, T], out=out)
    want, _ = slope.attn_varlen(xq.cuda(), xk.cuda(), xv.cuda(), [0, 15, T])
    assert torch.equal(out, want)
    pages = slope.KV4Cache(3, 16, 1, d, d)
    slope.kv4_write(pages, k, v, i32(list(range(T))))
    dense = slope.KV4Cache(3, 16, 1, d, d)
    slope.kv4_write(dense, xk.cuda(), xv.cuda(), i32(list(range(T))))
    assert torch.equal(torch.cat(slope.kv4_read(pages, i32(list(range(T))))), torch.cat(slope.kv4_read(dense, i32(list(range(T))))))


FIRST_CALLS = """
import torch, ring_attention_slope_gb300 as slope
q, k, v = (torch.randn(40, h, 64, device="cuda").bfloat16() for h in (8, 1, 1))
cache, slots = slope.KV4Cache(3, 16, 1, 64, 64), torch.arange(40, dtype=torch.int32, device="cuda")
table, lens = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3), torch.full((1,), 40, dtype=torch.int32, device="cuda")
def calls():
    qr, kr = slope.qk_norm_rope(q, k, rope=slope.Rope([0.5] * 32))
    out = slope.attn_varlen(qr, kr, v, [0, 15, 40])
    slope.kv4_write(cache, kr, v, slots)
    return (*out, *slope.kv4_read(cache, slots), *slope.kv4_attn(qr[39:], cache, table, lens))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
want = calls()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and slope.device_status() == (0, 0)
"""


def test_first_calls_of_a_process_are_captured():
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=Path(__file__).resolve().parents[1], timeout=100,
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]


# ---------------------------------------------------------------- packed prompts

OUT_MAX, OUT_REL_L2, LSE_MAX = 2e-2, 5e-3, 1e-3  # as the prefill attention's parity tests


def check_varlen(q, k, v, cu, window=0, causal=True, out_dtype=None, scale=0.0, heads=None):
    out, lse = slope.attn_varlen(q.cuda(), k.cuda(), v.cuda(), cu, causal=causal, window=window, out_dtype=out_dtype,
                                 scale=scale)
    og, lg = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    for a, e in zip(cu[:-1], cu[1:]):
        if a == e:
            continue
        ro, rl = oracle.attention(q[a:e], k[a:e], v[a:e], causal=causal, window=window, scale=scale or None, heads=heads)
        o, le = (og[a:e], lg[:, a:e]) if heads is None else (og[a:e][:, heads], lg[heads][:, a:e])
        assert np.isfinite(o).all()
        assert np.max(np.abs(le - rl)) <= LSE_MAX, (a, e, np.max(np.abs(le - rl)))
        assert np.max(np.abs(o - ro)) <= OUT_MAX, (a, e, np.max(np.abs(o - ro)))
        assert np.linalg.norm(o - ro) <= OUT_REL_L2 * np.linalg.norm(ro), (a, e)
    return out, lse


def packed(lens, Hq, H, dqk, dv, seed, lead=0, tail=0):
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    T = cu[-1] + tail
    s = 0.7
    return rand(T, Hq, dqk, seed=seed, scale=s), rand(T, H, dqk, seed=seed + 1, scale=s), rand(T, H, dv, seed=seed + 2, scale=s), cu


@pytest.mark.parametrize("lens", [[1], [5, 1, 0, 16, 17], [127, 128, 129], [300, 2, 515], [1] * 70, [0, 0, 33, 0],
                                  [(7 * i) % 23 for i in range(300)]])
@pytest.mark.parametrize("Hq,H", [(8, 1), (4, 4), (6, 2), (12, 2)])
def test_varlen_lengths(lens, Hq, H):
    check_varlen(*packed(lens, Hq, H, 64, 64, 140))


@pytest.mark.parametrize("dqk,dv", [(64, 64), (64, 128), (128, 64), (128, 128), (192, 64), (192, 128)])
@pytest.mark.parametrize("Hq,H", [(2, 2), (16, 2), (5, 1), (64, 1)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_varlen_sizes(dqk, dv, Hq, H, out_dtype):
    check_varlen(*packed([40, 200, 3, 385], Hq, H, dqk, dv, 150), out_dtype=out_dtype)


@pytest.mark.parametrize("window,causal", [(1, True), (30, True), (128, True), (300, True), (5000, True), (0, False), (60, False)])
@pytest.mark.parametrize("dqk,dv,Hq,H", [(64, 64, 8, 1), (64, 64, 3, 3), (192, 128, 2, 2), (128, 128, 8, 2),
                                        (192, 64, 2, 2)])
def test_varlen_masks(window, causal, dqk, dv, Hq, H):
    check_varlen(*packed([40, 333, 130, 700], Hq, H, dqk, dv, 160), window=window, causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[180] * 30, [256] * 24, [117, 353, 588] * 6, [150, 1] * 36])
def test_varlen_many_middling(lens, causal):
    """Enough short work tiles of 64-wide heads that two Q tiles share a CTA, with NaN behind the last sequence."""
    q, k, v, cu = packed(lens, 16, 2, 64, 64, 168, lead=3, tail=20)
    for x in (q, k, v):
        x[:3] = x[cu[-1]:] = float("nan")
    check_varlen(q, k, v, cu, causal=causal, heads=[0, 7, 8, 15])


@pytest.mark.parametrize("dqk,dv", [(64, 64), (128, 128), (192, 64), (192, 128)])
def test_varlen_second_tile_starts_at_a_sequence_end(dqk, dv):
    """A CTA's second Q tile whose first step is the last, partial one, many times over: the V rows that it clears are
    those of that step and not of the one before."""
    lens = [129 + i % 40 for i in range(100)]
    q, k, v, cu = packed(lens, 2, 2, dqk, dv, 165)
    for window in (2, 20):
        check_varlen(q, k, v, cu, window=window)


@pytest.mark.parametrize("dqk,dv,Hq,H,window", [(64, 64, 8, 1, 0), (64, 64, 8, 1, 50), (64, 64, 1, 1, 0), (192, 128, 2, 2, 0),
                                               (128, 128, 4, 1, 0), (64, 128, 2, 2, 40)])
def test_varlen_what_lies_outside_does_not_leak(dqk, dv, Hq, H, window):
    """NaN before, after and in a sequence of its own between the others; rows outside stay as they were."""
    lens = [30, 21, 200, 140]
    q, k, v, cu = packed(lens, Hq, H, dqk, dv, 170, lead=7, tail=50)
    bad = list(range(0, 7)) + list(range(cu[1], cu[2])) + list(range(cu[4], cu[4] + 50))
    for x in (q, k, v):
        x[bad] = math.nan
    v[bad[::2]] = math.inf
    T = q.shape[0]
    out = torch.full((T, Hq, dv), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, T), 5.0, device="cuda")
    slope.attn_varlen(q.cuda(), k.cuda(), v.cuda(), cu, window=window, out=out, lse=lse)
    for i in (0, 2, 3):
        a, e = cu[i], cu[i + 1]
        ro, rl = oracle.attention(q[a:e], k[a:e], v[a:e], causal=True, window=window)
        assert np.max(np.abs(out[a:e].float().cpu().double().numpy() - ro)) <= OUT_MAX, i
        assert np.max(np.abs(lse[:, a:e].cpu().double().numpy() - rl)) <= LSE_MAX, i
    outside = list(range(0, cu[0])) + list(range(cu[-1], T))
    assert (out[outside] == 5).all() and (lse[:, outside] == 5).all()


def test_varlen_strides():
    lens, Hq, H, d = [100, 31], 4, 2, 64
    q, k, v, cu = packed(lens, Hq, H, d, d, 180)
    T = q.shape[0]
    buf = torch.zeros(T, Hq + 2 * H + 1, d + 8, dtype=torch.bfloat16, device="cuda")
    views = [buf[:, 0:Hq, :d], buf[:, Hq:Hq + H, 8:], buf[:, Hq + H:Hq + 2 * H, :d]]
    for x, y in zip((q, k, v), views):
        y.copy_(x.cuda())
    ref, rl = slope.attn_varlen(q.cuda(), k.cuda(), v.cuda(), cu)
    obuf = torch.full((T, Hq + 1, d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((T, 3 * Hq), 3.0, device="cuda")
    slope.attn_varlen(*views, cu, out=obuf[:, 1:, 8:], lse=lbuf[:, ::3].t())
    assert torch.equal(obuf[:, 1:, 8:], ref) and torch.equal(lbuf[:, ::3].t(), rl)
    assert (obuf[:, 0] == 3).all() and (obuf[:, :, :8] == 3).all() and (lbuf[:, 1::3] == 3).all()


def test_varlen_one_sequence_is_the_prefill_attention():
    q, k, v, cu = packed([1500], 8, 2, 64, 64, 190)
    out, lse = slope.attn_varlen(q.cuda(), k.cuda(), v.cuda(), cu)
    ref, rl = slope.attn_partial(q.cuda(), k.cuda(), v.cuda(), out_dtype=torch.bfloat16)
    assert (out.float() - ref.float()).abs().max() <= 2.0 ** -7 * ref.float().abs().max()
    assert (lse - rl).abs().max() <= 1e-5 * rl.abs().max()


def test_varlen_captured():
    q, k, v, cu = packed([70, 300, 9] * 15, 8, 1, 64, 64, 200)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    ref, rl = slope.attn_varlen(q, k, v, cu)
    out, lse = torch.zeros_like(ref), torch.zeros_like(rl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slope.attn_varlen(q, k, v, cu, out=out, lse=lse)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, rl)


# ---------------------------------------------------------------- together

def test_prompts_then_decode_as_a_server_runs_them():
    """Two packed prompts are normed, rotated, attended and cached; then each gets one more token, whose attention over
    the cache equals the prefill attention over the rows read back, in one piece and merged from two."""
    Hq, H, d, page, lens = 8, 2, 64, 32, [75, 33]
    cu = [0, 75, 108]
    dev = "cuda"
    freq, _ = slope.rope_inv_freq(d, 10000.0, scaling="bands", factor=8, original=8192, fast=4, slow=1)
    rope = slope.Rope(freq)
    qw, kw = rand(d, seed=300, dtype=torch.float32).to(dev), rand(d, seed=301, dtype=torch.float32).to(dev)
    pos = i32(list(range(75)) + list(range(33)))
    q, k, v = rand(108, Hq, d, seed=302).to(dev), rand(108, H, d, seed=303).to(dev), rand(108, H, d, seed=304).to(dev)
    q, k = slope.qk_norm_rope(q, k, q_weight=qw, k_weight=kw, rope=rope, positions=pos)
    out, lse = slope.attn_varlen(q, k, v, cu)
    for a, e in ((0, 75), (75, 108)):
        o, l = slope.attn_partial(q[a:e], k[a:e], v[a:e], out_dtype=torch.bfloat16)
        assert (out[a:e].float() - o.float()).abs().max() <= OUT_MAX and (lse[:, a:e] - l).abs().max() <= LSE_MAX

    cache = slope.KV4Cache(9, page, H, d, d)
    table = i32([[4, 0, 7, 2], [8, 1, 5, 3]])
    slot = lambda b, t: table[b, t // page].long() * page + t % page  # noqa: E731
    t = [torch.arange(n, device=dev) for n in lens]
    slope.kv4_write(cache, k, v, torch.cat([slot(0, t[0]), slot(1, t[1])]).int())
    # the next token of both
    q1, k1, v1 = rand(2, Hq, d, seed=305).to(dev), rand(2, H, d, seed=306).to(dev), rand(2, H, d, seed=307).to(dev)
    q1, k1 = slope.qk_norm_rope(q1, k1, q_weight=qw, k_weight=kw, rope=rope, positions=i32(lens))
    new = torch.stack([slot(b, torch.tensor(n, device=dev)) for b, n in enumerate(lens)]).int()
    slope.kv4_write(cache, k1, v1, new)
    kv_lens = i32([n + 1 for n in lens])
    out1, lse1 = slope.kv4_attn(q1, cache, table, kv_lens, out_dtype=torch.float32)
    for b, n in enumerate(lens):
        all_slots = slot(b, torch.arange(n + 1, device=dev)).int()
        kr, vr = slope.kv4_read(cache, all_slots)
        o, l = slope.attn_partial(q1[b:b + 1], kr, vr, q_off=n)
        # both round their weights to bf16, and the prefill attention its keys and values too
        assert (o - out1[b:b + 1]).abs().max() <= OUT_MAX and (l - lse1[:, b:b + 1]).abs().max() <= 5e-2
        # the cache without the new token, merged with the new token's own partial
        oc, lc = slope.kv4_attn(q1[b:b + 1], cache, table[b:b + 1], i32([n]), out_dtype=torch.float32)
        ot, lt = slope.attn_partial(q1[b:b + 1], kr[n:], vr[n:], q_off=n, kv_off=n)
        om, lm = slope.lse_merge([oc, ot], [lc, lt], out_dtype=torch.float32)
        assert (om - out1[b:b + 1]).abs().max() <= OUT_MAX and (lm - lse1[:, b:b + 1]).abs().max() <= 5e-2
