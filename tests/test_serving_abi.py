"""The serving calls' exports, structures and refusals: every argument error is reported before anything touches
the GPU (these run without one, on descriptors whose addresses are never read)."""
import ctypes
import math
import os
import re
import subprocess

import pytest

import ring_attention_slope_gb300 as slope
from _lib import ROOT, built_lib

S_OK, E_NULL, E_DTYPE, E_SHAPE, E_STRIDE, E_LAYOUT, E_UNSUP, E_WS = 0, -1, -2, -3, -4, -5, -8, -9
BF16, F32 = 0, 1
HEADER = os.path.join(ROOT, "include", "slope_serving.h")


@pytest.fixture(scope="module")
def lib():
    return built_lib()


def t(shape, dtype=BF16, data=0x10000, stride=None):
    d = slope.SlopeTensor()
    d.data, d.dtype, d.ndim = data, dtype, len(shape)
    if stride is None:
        stride = [math.prod(shape[i + 1:]) for i in range(len(shape))]
    for i, s in enumerate(shape):
        d.shape[i], d.stride[i] = s, stride[i]
    return d


def ref(d):
    return ctypes.byref(d) if d is not None else None


def test_exports_every_declared_symbol(lib):
    names = sorted(set(re.findall(r"SLOPE_API\s+[\w\s\*]+?\b(slope_\w+)\s*\(", open(HEADER).read())))
    assert names == sorted(slope.EXPORTED_SERVING)
    for n in names:
        assert hasattr(lib, n), n


def test_header_compiles_as_c99_and_matches_the_binding(tmp_path):
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    fields = [(s, f) for s, c in (("slope_rope", slope.SlopeRope), ("slope_kv4_cache", slope.SlopeKV4Cache)) for f, _ in c._fields_]
    lines = "".join(f'printf("%zu %zu\\n", offsetof({s}, {f}), sizeof((({s}*)0)->{f}));\n' for s, f in fields)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "slope_serving.h"\nint main(void) {\n' + lines +
                   'printf("%zu %zu\\n", sizeof(slope_rope), sizeof(slope_kv4_cache));\n'
                   'printf("%d %d\\n", SLOPE_ROPE_YARN, SLOPE_KV4_MAX_Q_LEN);\nreturn 0; }\n')
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.dirname(HEADER),
                           str(src), "-o", str(exe)])
    got = [tuple(int(x) for x in line.split()) for line in subprocess.check_output([str(exe)], text=True).splitlines()]
    cls = {"slope_rope": slope.SlopeRope, "slope_kv4_cache": slope.SlopeKV4Cache}
    # the packed forms that the binding passes are the same bytes
    freq = (ctypes.c_double * 8)()
    packed = slope.serving._pack_rope(3, 16, 1, 0.5, ctypes.addressof(freq))
    assert packed == bytes(slope.SlopeRope(3, 16, 1, 0.5, freq))
    assert slope.serving._pack_cache(4096, 7, 64, 2, 128, 64) == bytes(slope.SlopeKV4Cache(4096, 7, 64, 2, 128, 64))
    for (s, f), have in zip(fields, got):
        field = getattr(cls[s], f)
        assert have == (field.offset, field.size), (s, f)
    assert got[-2] == (ctypes.sizeof(slope.SlopeRope), ctypes.sizeof(slope.SlopeKV4Cache))
    assert got[-1] == (4, 64)


# ---------------------------------------------------------------- frequencies

def inv_freq(lib, dim, base=10000.0, kind=0, factor=1.0, original=0.0, fast=0.0, slow=0.0):
    out, att = (ctypes.c_double * max(1, dim // 2 + 1))(), ctypes.c_double()
    st = lib.slope_rope_inv_freq(dim, base, kind, factor, original, fast, slow, out, ctypes.byref(att))
    return st, list(out)[:max(0, dim // 2)], att.value


def test_inv_freq_formulas(lib):
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    close = lambda a, b: all(abs(x - y) <= 1e-14 * abs(y) for x, y in zip(a, b)) and len(a) == len(b)  # noqa: E731
    assert inv_freq(lib, 64)[0] == S_OK and close(inv_freq(lib, 64)[1], plain) and inv_freq(lib, 64)[2] == 1
    assert close(inv_freq(lib, 64, kind=1, factor=4)[1], [f / 4 for f in plain])
    ntk = inv_freq(lib, 64, kind=2, factor=4)[1]
    assert ntk[0] == 1 and abs(ntk[31] - plain[31] / 4) <= 1e-14 * plain[31]
    bands = inv_freq(lib, 64, kind=3, factor=8, original=8192, fast=4, slow=1)
    assert bands[0] == S_OK and bands[2] == 1
    for f, b in zip(plain, bands[1]):
        turns = 8192 * f / (2 * math.pi)
        keep = min(1, max(0, (turns - 1) / 3))
        assert abs(b - (keep * f + (1 - keep) * f / 8)) <= 1e-14 * f
        assert turns < 4 or b == f
        assert turns > 1 or abs(b - f / 8) <= 1e-15 * f
    st, yarn, att = inv_freq(lib, 64, kind=4, factor=16, original=4096, fast=32, slow=1)
    assert st == S_OK and abs(att - (0.1 * math.log(16) + 1)) < 1e-15
    at = lambda n: 64 * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(10000))  # noqa: E731
    lo, hi = math.floor(at(32)), math.ceil(at(1))
    for i, (f, y) in enumerate(zip(plain, yarn)):
        s = min(1, max(0, (i - lo) / (hi - lo)))
        assert abs(y - (f * (1 - s) + f / 16 * s)) <= 1e-14 * f


def test_inv_freq_refusals(lib):
    ok = dict(kind=4, factor=8, original=4096, fast=32, slow=1)
    assert inv_freq(lib, 64, **ok)[0] == S_OK
    for bad in (dict(factor=0.5), dict(factor=math.nan), dict(original=0), dict(fast=1), dict(slow=0), dict(fast=math.inf),
                dict(base=1.0), dict(base=math.inf), dict(base=math.nan)):
        assert inv_freq(lib, 64, **{**ok, **bad})[0] == E_SHAPE, bad
    for dim in (0, 2, 3, 65, 514, -4):
        assert inv_freq(lib, dim)[0] == E_SHAPE, dim
    assert inv_freq(lib, 64, kind=5)[0] == E_UNSUP and inv_freq(lib, 64, kind=-1)[0] == E_UNSUP
    assert lib.slope_rope_inv_freq(64, 10000.0, 0, 1, 0, 0, 0, None, None) == E_NULL
    assert lib.slope_rope_inv_freq(64, 10000.0, 0, 1, 0, 0, 0, (ctypes.c_double * 32)(), None) == S_OK


# ---------------------------------------------------------------- norm and rotation

def rope(dim=64, begin=0, factor=1.0, freq=None, null=False):
    freq = [1.0] * (dim // 2) if freq is None else freq
    return slope.SlopeRope(begin, dim, 0, factor, None if null else (ctypes.c_double * len(freq))(*freq))


def norm_rope(lib, q=None, k=None, qw=None, kw=None, norm=1, eps=1e-6, r=None, pos=None, pos0=0, qo=None, ko=None):
    return lib.slope_qk_norm_rope(ref(q), ref(k), ref(qw), ref(kw), norm, eps, ref(r), pos, pos0,
                                  ref(qo), ref(ko), None)


def test_norm_rope_refusals(lib):
    T, Hq, Hkv, d = 0, 8, 2, 64  # no tokens: what is accepted does nothing
    base = dict(q=t([T, Hq, d]), k=t([T, Hkv, d]), qo=t([T, Hq, d]), ko=t([T, Hkv, d]), r=rope())

    def call(**kw):
        return norm_rope(lib, **{**base, **kw})

    assert call() == S_OK and call(k=None, ko=None) == S_OK and call(q=None, qo=None) == S_OK
    assert call(qw=t([1, d], F32), kw=t([Hkv, d], BF16)) == S_OK
    assert norm_rope(lib) == E_NULL and call(qo=None) == E_NULL and call(k=None) == E_NULL
    assert call(k=None, ko=None, kw=t([1, d])) == E_NULL
    assert call(q=t([T, Hq, d], 3)) == E_DTYPE and call(qo=t([T, Hq, d], F32)) == E_DTYPE       # q and k outputs differ
    assert call(q=t([T, Hq, d], F32)) == E_DTYPE                                                # q and k differ
    assert call(q=t([T, Hq, 96]), qo=t([T, Hq, 96])) == E_UNSUP
    assert call(qo=t([T, Hq + 1, d])) == E_SHAPE and call(q=t([Hq, d]), qo=t([Hq, d])) == E_SHAPE
    assert call(k=t([T, Hkv, 128]), ko=t([T, Hkv, 128])) == E_SHAPE
    assert call(qw=t([1, d + 1], F32)) == E_SHAPE and call(qw=t([3, d], F32)) == E_SHAPE
    assert call(qw=t([1, d], 7)) == E_DTYPE and call(qw=t([1, d], F32, data=0)) == E_NULL
    assert call(qw=t([1, d], F32, stride=[d, 2])) == E_STRIDE and call(qw=t([1, d], F32, data=0x10002)) == E_STRIDE
    assert call(norm=0, qw=t([1, d], F32)) == E_UNSUP and call(norm=0) == S_OK
    assert call(eps=-1.0) == E_SHAPE and call(eps=math.nan) == E_SHAPE and call(eps=math.inf) == E_SHAPE
    for bad in (rope(dim=8), rope(dim=24, freq=[1.0] * 12), rope(dim=80, freq=[1.0] * 40), rope(dim=32, begin=40),
                rope(dim=32, begin=4), rope(dim=32, begin=-8), rope(factor=math.inf), rope(freq=[math.nan] * 32)):
        assert call(r=bad) == E_SHAPE
    assert call(r=rope(null=True)) == E_NULL
    assert call(pos0=2 ** 31 + 1) == E_SHAPE and call(pos0=-(2 ** 31) - 1) == E_SHAPE and call(pos0=2 ** 31) == S_OK
    # strides and pointers, with tokens
    n = 4
    full = dict(q=t([n, Hq, d]), k=None, qo=t([n, Hq, d], data=0x90000), ko=None)
    assert call(**{**full, "q": t([n, Hq, d], stride=[Hq * d + 4, d, 1])}) == E_STRIDE
    assert call(**{**full, "q": t([n, Hq, d], stride=[Hq * d, d, 2])}) == E_STRIDE
    assert call(**{**full, "qo": t([n, Hq, d], data=0x90008)}) == E_STRIDE
    assert call(**{**full, "q": t([n, Hq, d], data=0)}) == E_NULL
    assert call(**full, pos=0x70002) == E_STRIDE
    same = t([n, Hq, d])
    assert call(**{**full, "q": same, "qo": t([n, Hq, d], stride=[2 * Hq * d, d, 1])}) == E_STRIDE  # not in place
    assert call(**{**full, "q": same, "qo": t([n, Hq, d], F32)}) == E_STRIDE


# ---------------------------------------------------------------- packed prompts

def test_varlen_refusals(lib):
    T, Hq, H, d = 100, 8, 2, 64
    base = dict(q=t([T, Hq, d]), k=t([T, H, d]), v=t([T, H, d]), out=t([T, Hq, d]), lse=t([Hq, T], F32), cu=[5, 5],
                n=None, window=0)

    def call(**kw):
        a = {**base, **kw}
        cu = (ctypes.c_int64 * len(a["cu"]))(*a["cu"]) if a["cu"] is not None else None
        n = len(a["cu"]) - 1 if a["n"] is None else a["n"]
        return lib.slope_attn_varlen(ref(a["q"]), ref(a["k"]), ref(a["v"]), cu, n, 1, a["window"], 0.0, ref(a["out"]),
                                     ref(a["lse"]), None)

    assert call() == S_OK and call(cu=[0]) == S_OK and call(cu=[3, 3, 3, 3]) == S_OK  # nothing to do
    for cu in ([0, 101], [-1, 5], [0, 50, 49], [60, 30, 100]):
        assert call(cu=cu) == E_LAYOUT, cu
    assert call(cu=[0, 5], n=-1) == E_SHAPE and call(cu=None, n=2) == E_NULL
    assert call(q=None) == E_NULL and call(out=None) == E_NULL and call(lse=None) == E_NULL
    assert call(q=t([T, Hq, d], F32)) == E_DTYPE and call(lse=t([Hq, T], BF16)) == E_DTYPE
    assert call(k=t([T + 1, H, d])) == E_SHAPE and call(v=t([T, H + 1, d])) == E_SHAPE and call(k=t([T, H, 128])) == E_SHAPE
    assert call(k=t([T, 3, d]), v=t([T, 3, d])) == E_SHAPE
    assert call(q=t([T, Hq, 96]), k=t([T, H, 96])) == E_UNSUP
    assert call(window=-1) == E_SHAPE and call(window=(1 << 30) + 1) == E_SHAPE
    assert call(q=t([T, Hq, d], data=0x10008)) == E_STRIDE and call(q=t([T, Hq, d], stride=[Hq * d, d, 2])) == E_STRIDE
    assert call(out=t([T, Hq, d], stride=[Hq * d + 4, d, 1])) == E_STRIDE
    big = 1 << 28
    assert call(q=t([big, Hq, d]), k=t([big, H, d]), v=t([big, H, d]), out=t([big, Hq, d]), lse=t([Hq, big], F32)) == E_SHAPE


# ---------------------------------------------------------------- the cache

def cache(n_pages=4, page=64, H=2, dqk=64, dv=64, data=0x40000):
    return slope.SlopeKV4Cache(data, n_pages, page, H, dqk, dv)


BAD_CACHES = [(dict(dqk=96), E_UNSUP), (dict(dv=192), E_UNSUP), (dict(page=8), E_SHAPE), (dict(page=48), E_SHAPE),
              (dict(page=2048), E_SHAPE), (dict(n_pages=-1), E_SHAPE), (dict(H=0), E_SHAPE), (dict(H=65536), E_SHAPE),
              (dict(n_pages=2 ** 25), E_SHAPE), (dict(data=None), E_NULL), (dict(data=0x40008), E_STRIDE)]


def test_cache_sizes(lib):
    assert lib.slope_kv4_block_bytes(64, 64) == 1280 and lib.slope_kv4_block_bytes(192, 128) == 3200
    assert lib.slope_kv4_block_bytes(64, 192) == 0 and lib.slope_kv4_block_bytes(32, 64) == 0
    assert lib.slope_kv4_cache_bytes(10, 64, 8, 64, 64) == 10 * 4 * 8 * 1280
    assert lib.slope_kv4_cache_bytes(0, 64, 8, 64, 64) == 0 and lib.slope_kv4_cache_bytes(10, 63, 8, 64, 64) == 0
    assert lib.slope_kv4_cache_bytes(2 ** 20, 1024, 65535, 192, 128) == 2 ** 20 * 64 * 65535 * 3200  # past 2^32


def test_cache_store_refusals(lib):
    def both(c, k, v, slots=0x5000):
        w = lib.slope_kv4_write(ref(c), ref(k), ref(v), slots, None)
        r = lib.slope_kv4_read(ref(c), slots, ref(k), ref(v), None)
        assert w == r
        return w

    T, H = 7, 2
    k, v = t([T, H, 64]), t([T, H, 64])
    for kw, status in BAD_CACHES:
        assert both(cache(**kw), k, v) == status, kw
    assert both(None, k, v) == E_NULL and both(cache(), None, v) == E_NULL and both(cache(), k, None) == E_NULL
    assert both(cache(), k, v, slots=None) == E_NULL and both(cache(), k, v, slots=0x5002) == E_STRIDE
    assert both(cache(), t([T, H, 64], F32), v) == E_DTYPE and both(cache(), t([T, H, 64], 4), v) == E_DTYPE
    assert both(cache(), t([T, H + 1, 64]), v) == E_SHAPE and both(cache(), k, t([T + 1, H, 64])) == E_SHAPE
    assert both(cache(dqk=128), k, v) == E_SHAPE and both(cache(dv=128), k, v) == E_SHAPE
    assert both(cache(), t([T, H, 64], stride=[H * 64 + 4, 64, 1]), v) == E_STRIDE
    assert both(cache(), k, t([T, H, 64], stride=[H * 64, 64, 2])) == E_STRIDE
    assert both(cache(), t([T, H, 64], data=0x10008), v) == E_STRIDE and both(cache(), t([T, H, 64], data=0), v) == E_NULL
    none = t([0, H, 64], data=0)
    assert both(cache(), none, none, slots=None) == S_OK
    assert both(cache(n_pages=0, data=None), none, none) == S_OK


def test_cache_attention_refusals(lib):
    B, Hq, H, d = 3, 8, 2, 64
    base = dict(q=t([B, Hq, d]), c=cache(), table=0x6000, stride=5, pages=5, lens=0x7000, q_len=1, window=0,
                out=t([B, Hq, d]), lse=t([Hq, B], F32), ws=0x100000, n=1 << 30)

    def call(**kw):
        a = {**base, **kw}
        return lib.slope_kv4_attn(ref(a["q"]), ref(a["c"]), a["table"], a["stride"], a["pages"], a["lens"], a["q_len"],
                                  a["window"], 0.0, ref(a["out"]), ref(a["lse"]), a["ws"], a["n"], None)

    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    assert call(q=None) == E_NULL and call(out=None) == E_NULL and call(table=None) == E_NULL and call(lens=None) == E_NULL
    assert call(q=t([B, Hq, d], F32)) == E_DTYPE and call(lse=t([Hq, B], BF16)) == E_DTYPE
    assert call(q_len=0) == E_SHAPE and call(q_len=2) == E_SHAPE and call(q_len=-1) == E_SHAPE
    assert call(q=t([130, Hq, d]), out=t([130, Hq, d]), lse=t([Hq, 130], F32), q_len=65) == E_UNSUP
    assert call(q=t([65536, Hq, d]), out=t([65536, Hq, d]), lse=t([Hq, 65536], F32)) == E_SHAPE
    assert call(q=t([B, 7, d]), out=t([B, 7, d]), lse=t([7, B], F32)) == E_SHAPE              # 7 query heads on 2
    assert call(q=t([B, Hq, 128])) == E_SHAPE and call(out=t([B, Hq, 128])) == E_SHAPE
    assert call(window=-1) == E_SHAPE and call(stride=4) == E_SHAPE and call(pages=-1) == E_SHAPE
    assert call(pages=1 << 22, stride=1 << 22) == E_SHAPE                                        # 2^28 positions
    assert call(q=t([B, Hq, d], data=0x10008)) == E_STRIDE and call(q=t([B, Hq, d], stride=[Hq * d + 4, d, 1])) == E_STRIDE
    assert call(out=t([B, Hq, d], stride=[Hq * d + 2, d, 1])) == E_STRIDE and call(table=0x6002) == E_STRIDE
    need = lib.slope_kv4_attn_workspace_size(B, Hq, ref(cache()), 1)
    assert need > 0 and call(n=need - 1) == E_WS and call(ws=None) == E_WS and call(ws=0x100010) == E_WS
    assert call(q=t([0, Hq, d], data=0), out=t([0, Hq, d], data=0), lse=t([Hq, 0], F32, data=0, stride=[1, 1]), ws=None) == S_OK


def test_cache_attention_workspace_size(lib):
    size = lambda B, Hq, q_len, **kw: lib.slope_kv4_attn_workspace_size(B, Hq, ref(cache(**kw)), q_len)  # noqa: E731
    assert size(1, 8, 1) == size(60000, 8, 1)      # the split is by CTAs, whatever the batch
    assert size(1, 8, 3) > size(1, 8, 2) == size(1, 2, 8) and size(1, 8, 1, dv=128) > size(1, 8, 1)
    for bad in (size(-1, 8, 1), size(65536, 8, 1), size(1, 7, 1), size(1, 0, 1), size(1, 8, 0), size(1, 8, 65),
                size(1, 8, 1, dqk=32), lib.slope_kv4_attn_workspace_size(1, 8, None, 1)):
        assert bad == 0
