"""The calls on the 16-bit paged cache: exports, structures and refusals, of the C ABI and of the binding.  Every argument
error is reported before anything touches the GPU (these run without one: addresses are never read)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import ring_attention_slope_gb300 as slope
from _lib import ROOT, built_lib
from test_serving_abi import (BF16, E_DTYPE, E_NULL, E_SHAPE, E_STRIDE, E_UNSUP, E_WS, F32, S_OK, ref, t)
from test_serving_marshal import Fake, i32

HEADER = os.path.join(ROOT, "include", "slope_kv.h")


@pytest.fixture(scope="module")
def lib():
    return built_lib()


@pytest.fixture(scope="module")
def m():
    built_lib()
    return slope.kv._bound()


def test_exports_every_declared_symbol(lib):
    names = sorted(set(re.findall(r"SLOPE_API\s+[\w\s\*]+?\b(slope_\w+)\s*\(", open(HEADER).read())))
    assert names == sorted(slope.EXPORTED_KV)
    for n in names:
        assert hasattr(lib, n), n


def test_header_compiles_as_c99_and_matches_the_binding(tmp_path):
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    cls = {"slope_kv_cache": slope.SlopeKVCache, "slope_kv_batch": slope.SlopeKVBatch}
    fields = [(s, f) for s, c in cls.items() for f, _ in c._fields_]
    lines = "".join(f'printf("%zu %zu\\n", offsetof({s}, {f}), sizeof((({s}*)0)->{f}));\n' for s, f in fields)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "slope_kv.h"\nint main(void) {\n' + lines +
                   'printf("%zu %zu\\n", sizeof(slope_kv_cache), sizeof(slope_kv_batch));\nreturn 0; }\n')
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.dirname(HEADER),
                           str(src), "-o", str(exe)])
    got = [tuple(int(x) for x in line.split()) for line in subprocess.check_output([str(exe)], text=True).splitlines()]
    for (s, f), have in zip(fields, got):
        field = getattr(cls[s], f)
        assert have == (field.offset, field.size), (s, f)
    assert got[-1] == (ctypes.sizeof(slope.SlopeKVCache), ctypes.sizeof(slope.SlopeKVBatch))
    packed = slope.kv._pack_cache(4096, 8192, 7, 64, 2, 128, 64, 1, 2, 3, 4, 5, 6)
    three = ctypes.c_int64 * 3
    assert packed == bytes(slope.SlopeKVCache(4096, 8192, 7, 64, 2, 128, 64, three(1, 2, 3), three(4, 5, 6)))


# ---------------------------------------------------------------- the C ABI

def cache(n_pages=4, page=64, H=2, dqk=64, dv=64, k=0x40000, v=0x80000, ks=None, vs=None):
    three = ctypes.c_int64 * 3
    ks = ks or (H * page * dqk, page * dqk, dqk)
    vs = vs or (H * page * dv, page * dv, dv)
    return slope.SlopeKVCache(k, v, n_pages, page, H, dqk, dv, three(*ks), three(*vs))


BAD_CACHES = [(dict(dqk=96), E_UNSUP), (dict(dv=192), E_UNSUP), (dict(page=8), E_SHAPE), (dict(page=48), E_SHAPE),
              (dict(page=2048), E_SHAPE), (dict(n_pages=0), E_SHAPE), (dict(n_pages=-1), E_SHAPE), (dict(H=0), E_SHAPE),
              (dict(H=65536), E_SHAPE), (dict(n_pages=2 ** 25), E_SHAPE), (dict(k=None), E_NULL), (dict(v=None), E_NULL),
              (dict(k=0x40008), E_STRIDE), (dict(v=0x40002), E_STRIDE), (dict(ks=(8192, 4096, 60)), E_STRIDE),
              (dict(vs=(0, 4096, 64)), E_STRIDE), (dict(ks=(8192, -64, 64)), E_STRIDE),
              (dict(vs=(2 ** 39, 4096, 64)), E_STRIDE)]


def weights(c=None, **kw):
    c = c or cache()
    return t([c.n_pages, c.Hkv, c.page_size], **{"dtype": F32, **kw})


def test_write_refusals(lib):
    T, H = 7, 2
    k, v = t([T, H, 64]), t([T, H, 64])

    def call(c=None, k=k, v=v, slots=0x5000, w=None, **kw):
        return lib.slope_kv_write(ref(c or cache(**kw)), ref(k), ref(v), slots, ref(w), None)

    for kw, status in BAD_CACHES:
        assert call(**{"c": cache(**kw)}) == status, kw
    assert lib.slope_kv_write(None, ref(k), ref(v), 0x5000, None, None) == E_NULL
    assert call(k=None) == E_NULL and call(v=None) == E_NULL and call(slots=None) == E_NULL and call(slots=0x5002) == E_STRIDE
    assert call(k=t([T, H, 64], F32)) == E_DTYPE and call(k=t([T, H, 64], 4), v=t([T, H, 64], 4)) == E_DTYPE
    assert call(k=t([T, H + 1, 64])) == E_SHAPE and call(v=t([T + 1, H, 64])) == E_SHAPE and call(k=t([T, 64])) == E_SHAPE
    assert call(c=cache(dqk=128)) == E_SHAPE and call(c=cache(dv=128)) == E_SHAPE
    assert call(k=t([T, H, 64], stride=[H * 64 + 4, 64, 1])) == E_STRIDE and call(v=t([T, H, 64], data=0x10008)) == E_STRIDE
    assert call(v=t([T, H, 64], stride=[H * 64, 64, 2])) == E_STRIDE and call(k=t([T, H, 64], data=0)) == E_NULL
    assert call(w=t([4, H, 64], BF16)) == E_DTYPE and call(w=t([4, H, 32], F32)) == E_SHAPE and call(w=t([H, 64], F32)) == E_SHAPE
    assert call(w=t([4, H, 64], F32, stride=[H * 64, 64, 2])) == E_STRIDE and call(w=t([4, H, 64], F32, data=0)) == E_NULL
    none = t([0, H, 64], data=0)
    assert call(k=none, v=none, slots=None) == S_OK and call(k=none, v=none, slots=None, w=weights()) == S_OK


BATCH = dict(B=3, cu_q=None, q_len=1, kv_lens=0x7000, block_table=0x6000, table_stride=5, max_pages=5)
BAD_BATCHES = [(dict(B=-1), E_SHAPE), (dict(B=65536, q_len=0), E_SHAPE), (dict(q_len=2), E_SHAPE), (dict(q_len=-1), E_SHAPE),
               (dict(max_pages=-1), E_SHAPE), (dict(table_stride=4), E_SHAPE), (dict(max_pages=1 << 22, table_stride=1 << 22), E_SHAPE),
               (dict(kv_lens=None), E_NULL), (dict(block_table=None), E_NULL), (dict(block_table=0x6002), E_STRIDE),
               (dict(kv_lens=0x7001), E_STRIDE), (dict(cu_q=0x9001), E_STRIDE)]


def batch(**kw):
    return slope.SlopeKVBatch(*{**BATCH, **kw}.values())


def both_attentions(lib, **kw):
    """Statuses of the attention and of the weights."""
    T, Hq, d = 3, 8, 64
    a = {**dict(q=t([T, Hq, d]), c=cache(), b=batch(), window=0, out=t([T, Hq, d]), lse=t([Hq, T], F32), w=weights(),
                ws=0x100000, n=1 << 40), **kw}
    return (lib.slope_kv_attn(ref(a["q"]), ref(a["c"]), ref(a["b"]), a["window"], 0.0, ref(a["out"]), ref(a["lse"]), a["ws"],
                              a["n"], None),
            lib.slope_kv_attn_weights(ref(a["q"]), ref(a["c"]), ref(a["b"]), ref(a["lse"]), a["window"], 0.0, 1, ref(a["w"]),
                                      a["ws"], a["n"], None))


def test_attention_refusals(lib):
    Hq, d = 8, 64

    def call(**kw):
        x, y = both_attentions(lib, **kw)
        assert x == y, kw
        return x

    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    for kw, status in BAD_BATCHES:
        assert call(b=batch(**kw)) == status, kw
    assert call(q=None) == E_NULL and call(b=None) == E_NULL and call(c=None) == E_NULL
    assert call(q=t([3, Hq, d], F32)) == E_DTYPE and call(lse=t([Hq, 3], BF16)) == E_DTYPE
    assert call(q=t([3, 7, d])) == E_SHAPE and call(q=t([3, Hq, 128])) == E_SHAPE and call(lse=t([Hq, 4], F32)) == E_SHAPE
    assert call(q=t([1 << 28, Hq, d])) == E_SHAPE and call(window=-1) == E_SHAPE and call(window=(1 << 30) + 1) == E_SHAPE
    assert call(q=t([3, Hq, d], data=0x10008)) == E_STRIDE and call(q=t([3, Hq, d], stride=[Hq * d + 4, d, 1])) == E_STRIDE
    assert call(q=t([3, Hq, d], stride=[1 << 39, d, 1])) == E_STRIDE and call(q=t([3, Hq, d], data=0)) == E_NULL
    assert call(n=16) == E_WS and call(ws=None) == E_WS and call(ws=0x100010) == E_WS
    assert call(q=t([0, Hq, d], data=0), b=batch(B=0), out=t([0, Hq, d], data=0), lse=t([Hq, 0], F32, data=0, stride=[1, 1]), ws=None) == S_OK
    # rows of no sequence only: nothing to do, or every weight 0
    assert both_attentions(lib, q=t([0, Hq, d], data=0), b=batch(q_len=0), out=t([0, Hq, d], data=0),
                           lse=t([Hq, 0], F32, data=0, stride=[1, 1]), ws=None) == (S_OK, S_OK)
    assert both_attentions(lib, out=None)[0] == E_NULL and both_attentions(lib, out=t([3, Hq, 128]))[0] == E_SHAPE
    assert both_attentions(lib, out=t([3, Hq, d], stride=[Hq * d + 4, d, 1]))[0] == E_STRIDE
    assert both_attentions(lib, out=t([3, Hq, d], data=0x10008))[0] == E_STRIDE
    assert both_attentions(lib, lse=None)[1] == E_NULL and both_attentions(lib, w=None)[1] == E_NULL
    assert both_attentions(lib, w=t([4, 2, 63], F32))[1] == E_SHAPE and both_attentions(lib, w=t([4, 2, 64], BF16))[1] == E_DTYPE


def test_workspace_sizes(lib):
    size = lambda T, Hq, q_len, **kw: lib.slope_kv_attn_workspace_size(T, Hq, ref(cache(**kw)), q_len)  # noqa: E731
    assert size(1, 8, 1) == size(1000, 8, 1)  # the split is by CTAs, whatever the batch
    assert size(1000, 8, 2) > size(1000, 8, 1) and size(1000, 8, 0) > size(1000, 8, 2) and size(1, 8, 1, dv=128) > 0
    need = size(3, 8, 1)
    assert need > 0 and both_attentions(lib, n=need - 1)[0] == E_WS
    w = lib.slope_kv_attn_weights_workspace_size(3, 8, ref(cache()), 1)
    assert w > 0 and both_attentions(lib, n=w - 1)[1] == E_WS
    for f in (lib.slope_kv_attn_workspace_size, lib.slope_kv_attn_weights_workspace_size):
        for bad in ((-1, 8, cache(), 1), (1 << 28, 8, cache(), 1), (1, 7, cache(), 1), (1, 0, cache(), 1), (1, 8, cache(), -1),
                    (1, 8, cache(dqk=32), 1), (1, 8, None, 1)):
            assert f(bad[0], bad[1], ref(bad[2]), bad[3]) == 0
    evict = lib.slope_kv_evict_workspace_size
    assert evict(2, 8, 1000) > evict(1, 8, 1000) > evict(1, 8, 10) > 0
    assert evict(-1, 8, 10) == evict(65536, 8, 10) == evict(1, 0, 10) == evict(1, 8, 0) == evict(1, 8, 1 << 28) == 0


def test_evict_refusals(lib):
    def call(**kw):
        a = {**dict(c=cache(), w=weights(), B=3, table=0x6000, stride=5, pages=5, lens=0x7000, keep=100, first=2, recent=20,
                    out_table=None, out_stride=0, out_pages=0, kept=0xa000, out_lens=0xb000, ws=0x100000, n=1 << 40), **kw}
        return lib.slope_kv_evict(ref(a["c"]), ref(a["w"]), a["B"], a["table"], a["stride"], a["pages"], a["lens"], a["keep"],
                                  a["first"], a["recent"], a["out_table"], a["out_stride"], a["out_pages"], a["kept"],
                                  a["out_lens"], a["ws"], a["n"], None)

    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    assert call(w=None) == E_NULL and call(w=t([4, 2, 64], BF16)) == E_DTYPE and call(w=t([3, 2, 64], F32)) == E_SHAPE
    assert call(B=-1) == E_SHAPE and call(B=65536) == E_SHAPE and call(stride=4) == E_SHAPE and call(pages=-1) == E_SHAPE
    assert call(lens=None) == E_NULL and call(table=None) == E_NULL and call(kept=None) == E_NULL and call(out_lens=None) == E_NULL
    for kw in (dict(keep=0), dict(keep=-1), dict(keep=1 << 28), dict(first=-1), dict(recent=-1), dict(first=90, recent=11),
               dict(first=101), dict(recent=1 << 62), dict(first=1 << 62)):
        assert call(**kw) == E_SHAPE, kw
    own = dict(out_table=0xc000, out_stride=2, out_pages=2)  # 128 positions
    assert call(**own, n=1) == E_WS                            # all else is right
    for kw in (dict(out_pages=1), dict(out_stride=1), dict(out_pages=-1), dict(out_pages=1 << 22, out_stride=1 << 22)):
        assert call(**{**own, **kw}) == E_SHAPE, kw
    assert call(**{**own, "out_table": 0xc002}) == E_STRIDE and call(kept=0xa001) == E_STRIDE and call(out_lens=0xb002) == E_STRIDE
    # no sequence can have more than the table's 320 tokens
    assert call(**own, keep=1000, n=1) == E_SHAPE and call(**{**own, "out_pages": 5, "out_stride": 5}, keep=1000, n=1) == E_WS
    need = lib.slope_kv_evict_workspace_size(3, 2, 100)
    assert call(n=1) == E_WS and need > 0 and call(ws=None) == E_WS and call(ws=0x100001) == E_WS
    assert call(B=0, table=None, lens=None, kept=None, ws=None) == S_OK


# ---------------------------------------------------------------- the binding

CACHE = slope.kv._pack_cache(0x40000, 0x80000, 4, 64, 2, 64, 64, 8192, 4096, 64, 8192, 4096, 64)


def test_binding_passes_what_it_is_given(m):
    f32 = lambda *s, **kw: Fake(s, torch.float32, **kw)  # noqa: E731
    k, w = Fake([3, 2, 64]), f32(4, 2, 64)
    none = Fake([0, 2, 64], ptr=0)
    assert m.kv_write(CACHE, none, none, i32(0, ptr=0), None, 0, 0) == S_OK
    assert m.kv_write(CACHE, none, none, i32(0, ptr=0), w, 0, 0) == S_OK
    assert m.kv_write(CACHE, k, Fake([3, 3, 64]), i32(3), w, 0, 0) == E_SHAPE
    assert m.kv_write(CACHE, k, k, i32(3), f32(4, 2, 64, stride=[128, 64, 2]), 0, 0) == E_STRIDE

    def attn(weights=False, **kw):
        a = {**dict(q=Fake([3, 8, 64]), table=i32(3, 5), lens=i32(3), cu=None, q_len=1, window=0, out=Fake([3, 8, 64]),
                    lse=f32(8, 3), w=w, ws=0x100000, n=0, cache=CACHE), **kw}
        head = (a["q"], a["cache"], a["table"], a["lens"], a["cu"], a["q_len"])
        if weights:
            return m.kv_attn_weights(*head, a["lse"], a["window"], 0.0, True, a["w"], a["ws"], a["n"], 0, 0)
        return m.kv_attn(*head, a["window"], 0.0, a["out"], a["lse"], a["ws"], a["n"], 0, 0)

    for kind in (False, True):
        call = lambda **kw: attn(kind, **kw)  # noqa: E731, B023
        assert call() == E_WS and call(cu=i32(4)) == E_WS and call(table=i32(3, 5, stride=[9, 1])) == E_WS  # all else is right
        assert call(q_len=2) == E_SHAPE and call(cu=i32(4), q_len=7) == E_WS  # row indices go before a length
        assert call(table=i32(3, 5, stride=[4, 1])) == E_SHAPE and call(window=-1) == E_SHAPE
        assert call(lens=i32(0, ptr=0), table=i32(0, 5), q=Fake([0, 8, 64], ptr=0), out=Fake([0, 8, 64], ptr=0),
                    lse=f32(8, 0, stride=[1, 1])) == S_OK
        for bad in (dict(table=i32(2, 5)), dict(table=i32(3)), dict(table=i32(3, 5, stride=[1, 3])), dict(lens=i32(3, 1)),
                    dict(cu=i32(3)), dict(cu=i32(5)), dict(lens=i32(3, stride=[2]))):
            with pytest.raises(ValueError):
                call(**bad)
        for bad in (dict(table=Fake([3, 5], torch.int64)), dict(lens=Fake([3])), dict(cu=Fake([4], torch.int64)),
                    dict(q_len=1.0), dict(cache=b"x")):
            with pytest.raises(TypeError):
                call(**bad)
        with pytest.raises(OverflowError):
            call(q_len=2 ** 31)
        with pytest.raises(ValueError):
            call(q=Fake([3, 8, 64], device=1))

    def evict(**kw):
        a = {**dict(w=w, table=i32(3, 5), lens=i32(3), keep=100, first=0, recent=0, out_table=None, kept=i32(3, 2, 100),
                    out_lens=i32(3), ws=0x100000, n=0), **kw}
        return m.kv_evict(CACHE, *a.values(), 0, 0)

    assert evict() == E_WS and evict(out_table=i32(3, 2)) == E_WS and evict(out_table=i32(3, 1)) == E_SHAPE
    assert evict(first=101) == E_SHAPE and evict(w=None) == E_NULL
    for bad in (dict(table=i32(2, 5)), dict(out_table=i32(2, 2)), dict(out_lens=i32(2))):
        with pytest.raises(ValueError):
            evict(**bad)
    with pytest.raises(TypeError):
        evict(kept=Fake([3, 2, 100], torch.int64))


def test_binding_counts_arguments(m):
    for f in (m.kv_write, m.kv_attn, m.kv_attn_weights, m.kv_evict, m.kv_attn_workspace_size, m.kv_evict_workspace_size):
        with pytest.raises(TypeError):
            f(1)


def test_cache_objects_refuse_what_does_not_fit():
    built_lib()
    make = lambda k, v: slope.KVCache(4, 16, 2, 64, 128, k=k, v=v)  # noqa: E731
    k, v = torch.empty(4, 2, 16, 64, dtype=torch.bfloat16), torch.empty(4, 2, 16, 128, dtype=torch.bfloat16)
    for a, b in ((k.float(), v), (k, v.half()), (v, v), (k, k), (k[:3], v), (k, v.transpose(1, 2))):
        with pytest.raises(TypeError):
            make(a, b)
    with pytest.raises(ValueError):
        make(k.transpose(2, 3).contiguous().transpose(2, 3), v)  # channels apart
    with pytest.raises(TypeError):
        make(k, v)  # right, but not on a GPU


def test_evict_workspace_holds_a_ticket_for_each_launch(lib):
    """A launch moves 512 sequences at most: its ticket, and a flag and two bounds for each of the pairs, have places of their own."""
    for B in (1, 512, 513, 32768, 32769, 65535):
        assert lib.slope_kv_evict_workspace_size(B, 1, 1) >= 4 * -(-B // 512) + 4 * B + 8 * B, B


def test_a_batch_with_row_indices_needs_the_workspace_of_any_length(lib):
    """What its longest run is, only the device knows."""
    rows = dict(q=t([32, 64, 64]), c=cache(H=8), out=t([32, 64, 64]), lse=t([64, 32], F32), w=weights(cache(H=8)))
    size = lambda q_len: lib.slope_kv_attn_workspace_size(32, 64, ref(cache(H=8)), q_len)  # noqa: E731
    assert size(4) < size(0)
    for n in (size(4), size(0) - 1):
        assert both_attentions(lib, **rows, b=batch(cu_q=0x9000, q_len=4), n=n)[0] == E_WS
    assert both_attentions(lib, **rows, b=batch(B=8, q_len=4), n=size(4) - 1)[0] == E_WS
