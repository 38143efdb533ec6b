"""The C module that makes descriptors of tensors: what it passes to the library and what it refuses.

It asks a tensor for a few attributes only, so plain objects with those stand in for CUDA tensors here (their
addresses are never read: every call ends in a refusal, or has no tokens)."""
import math

import pytest
import torch

import ring_attention_slope_gb300 as slope
from _lib import built_lib

S_OK, E_NULL, E_SHAPE, E_STRIDE, E_LAYOUT, E_UNSUP, E_WS = 0, -1, -3, -4, -5, -8, -9


class Fake:
    def __init__(self, shape, dtype=torch.bfloat16, stride=None, ptr=0x10000, device=0):
        self.shape, self.dtype, self.ptr, self.device_number = torch.Size(shape), dtype, ptr, device
        self._stride = tuple(stride) if stride else tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))

    def stride(self):
        return self._stride

    def data_ptr(self):
        return self.ptr

    def get_device(self):
        return self.device_number

    def numel(self):
        return math.prod(self.shape)


@pytest.fixture(scope="module")
def m():
    built_lib()
    return slope.serving._bound()


def i32(*shape, **kw):
    return Fake(shape, torch.int32, **kw)


CACHE = slope.serving._pack_cache(0x40000, 4, 64, 2, 64, 64)


def write(m, k=None, v=None, slots=None, cache=CACHE, T=3):
    return m.kv4_write(cache, k or Fake([T, 2, 64]), v or Fake([T, 2, 64]), slots or i32(T), 0, 0)


def test_descriptors_reach_the_library(m):
    """Shapes, strides, types and addresses: a refusal names the one that is wrong, and only that."""
    none = Fake([0, 2, 64], ptr=0)
    assert m.kv4_write(CACHE, none, none, i32(0, ptr=0), 0, 0) == S_OK
    assert m.kv4_read(CACHE, i32(0, ptr=0), none, none, 0, 0) == S_OK
    assert write(m, k=Fake([3, 3, 64])) == E_SHAPE and write(m, v=Fake([4, 2, 64])) == E_SHAPE
    assert write(m, k=Fake([3, 2, 64], stride=[132, 64, 1])) == E_STRIDE
    assert write(m, k=Fake([3, 2, 64], stride=[128, 64, 2])) == E_STRIDE
    assert write(m, v=Fake([3, 2, 64], ptr=0x10008)) == E_STRIDE
    assert write(m, k=Fake([3, 2, 64], torch.float32)) == -2  # k and v differ in type
    assert write(m, slots=i32(3, ptr=0x5002)) == E_STRIDE
    assert write(m, cache=slope.serving._pack_cache(0x40000, 4, 63, 2, 64, 64)) == E_SHAPE
    assert m.kv4_write(CACHE, None, Fake([3, 2, 64]), i32(0), 0, 0) == E_NULL


def test_norm_rope_arguments(m):
    q, k = Fake([0, 8, 64], ptr=0), Fake([0, 2, 64], ptr=0)
    rope = slope.Rope([1.0] * 32)._c

    def call(q=q, k=k, qw=None, kw=None, norm=True, eps=1e-6, rope=rope, pos=None, pos0=0, qo=q, ko=k):
        return m.qk_norm_rope(q, k, qw, kw, norm, eps, rope, pos, pos0, qo, ko, 0, 0)

    assert call() == S_OK and call(k=None, ko=None) == S_OK and call(pos=i32(0, ptr=0)) == S_OK
    # a vector of weights is [1, d]
    assert call(qw=Fake([64], torch.float32), kw=Fake([2, 64])) == S_OK
    assert call(qw=Fake([63])) == E_SHAPE and call(qw=Fake([64], stride=[2])) == E_STRIDE and call(kw=Fake([3, 64])) == E_SHAPE
    assert call(norm=False, qw=Fake([64])) == E_UNSUP and call(norm=0) == S_OK and call(eps=-1) == E_SHAPE
    assert call(rope=slope.Rope([1.0] * 32, begin=4)._c) == E_SHAPE and call(rope=None) == S_OK
    assert call(pos0=2 ** 31 + 1) == E_SHAPE
    # keys alone: one position for each of their rows
    alone = dict(q=None, qo=None, k=Fake([4, 2, 64], stride=[4, 64, 1]), ko=Fake([4, 2, 64]))
    assert call(**alone, pos=i32(4)) == E_STRIDE
    with pytest.raises(ValueError):
        call(**alone, pos=i32(0, ptr=0))
    for bad, error in ((dict(q=Fake([0, 64])), None), (dict(q=Fake([64])), ValueError), (dict(qw=Fake([1, 1, 1, 64])), ValueError),
                       (dict(pos=i32(1)), ValueError), (dict(pos=Fake([0], torch.int64)), TypeError), (dict(rope=b"x"), TypeError),
                       (dict(q=Fake([0, 8, 64], torch.float16)), TypeError), (dict(eps="1"), TypeError), (dict(pos0=1.5), TypeError),
                       (dict(pos0=2 ** 63), OverflowError), (dict(q=3), AttributeError)):
        if error is None:
            assert call(**bad) < 0
        else:
            with pytest.raises(error):
                call(**bad)
    with pytest.raises(TypeError):
        m.qk_norm_rope(q, k)


def test_devices(m):
    """A tensor elsewhere is refused, but for an empty one, and one that is no CUDA tensor."""
    with pytest.raises(ValueError):
        write(m, k=Fake([3, 2, 64], device=1))
    with pytest.raises(TypeError):
        write(m, v=Fake([3, 2, 64], device=-1))
    with pytest.raises(ValueError):
        write(m, slots=i32(3, device=1))
    none = Fake([0, 2, 64], ptr=0, device=-1)
    assert m.kv4_write(CACHE, none, none, i32(0, ptr=0, device=-1), 0, 0) == S_OK


def test_index_arrays(m):
    for slots in (i32(4), i32(3, 1), i32(3, stride=[2]), i32()):
        with pytest.raises(ValueError):
            write(m, slots=slots)
    with pytest.raises(TypeError):
        write(m, slots=Fake([3], torch.int64))


def test_varlen_lists(m):
    q, k = Fake([100, 8, 64]), Fake([100, 2, 64])
    lse = Fake([8, 100], torch.float32)

    def call(cu, **kw):
        a = {**dict(q=q, k=k, v=k, window=0, out=q, lse=lse), **kw}
        return m.attn_varlen(a["q"], a["k"], a["v"], cu, True, a["window"], 0.0, a["out"], a["lse"], 0, 0)

    assert call([5, 5]) == S_OK and call((3,)) == S_OK and call([7] * 400) == S_OK
    assert call([0, 101]) == E_LAYOUT and call([0] * 300 + [101]) == E_LAYOUT and call([4, 3]) == E_LAYOUT
    assert call([5, 5], window=-1) == E_SHAPE and call([5, 5], lse=None) == E_NULL
    for cu, error in (([], ValueError), (None, TypeError), ([0, "1"], TypeError), ([0, 1.0], TypeError), ([0, 2 ** 63], OverflowError)):
        with pytest.raises(error):
            call(cu)


def test_cache_attention_arguments(m):
    lse = Fake([8, 3], torch.float32)

    def call(**kw):
        a = {**dict(q=Fake([3, 8, 64]), table=i32(3, 5), lens=i32(3), q_len=1, window=0, out=Fake([3, 8, 64]), lse=lse,
                    ws=0x100000, n=0), **kw}
        return m.kv4_attn(a["q"], CACHE, a["table"], a["lens"], a["q_len"], a["window"], 0.0, a["out"], a["lse"], a["ws"],
                          a["n"], 0, 0)

    assert call() == E_WS and call(lse=None) == E_WS and call(table=i32(3, 5, stride=[9, 1])) == E_WS  # all else is right
    assert call(table=i32(3, 5, stride=[4, 1])) == E_SHAPE  # rows overlap
    assert call(q=Fake([0, 8, 64], ptr=0), table=i32(0, 5), lens=i32(0), out=Fake([0, 8, 64], ptr=0),
                lse=Fake([8, 0], torch.float32, stride=[1, 1]), q_len=5) == S_OK
    assert call(q=Fake([3, 7, 64]), out=Fake([3, 7, 64]), lse=None) == E_SHAPE
    for bad in (dict(q_len=2), dict(q_len=0), dict(q_len=2 ** 40), dict(table=i32(2, 5)), dict(table=i32(3)),
                dict(table=i32(3, 5, stride=[1, 3])), dict(lens=i32(2))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(table=Fake([3, 5], torch.int64)), dict(lens=Fake([3])), dict(q_len=1.0)):
        with pytest.raises(TypeError):
            call(**bad)


def test_no_reference_is_lost(m):
    """Calls that end well and calls that raise leave the reference counts of what they were given."""
    import sys

    k, slots, bad = Fake([3, 2, 64]), i32(3), Fake([3], torch.int64)
    things = [k, slots, bad, k.shape, k._stride, torch.bfloat16, torch.int32, CACHE]
    before = [sys.getrefcount(x) for x in things]
    for _ in range(50):
        assert write(m, k=k, slots=slots, v=Fake([4, 2, 64])) == E_SHAPE
        with pytest.raises(TypeError):
            write(m, k=k, slots=bad)
    assert [sys.getrefcount(x) for x in things] == before
