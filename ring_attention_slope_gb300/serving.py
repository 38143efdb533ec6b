"""The calls around the prefill attention (``include/slope_serving.h``): head norm with rotation, packed
prompts, the 4-bit paged key/value cache and attention over it.

Defaults and outputs are made here; the arguments go to the library through the C module ``_marshal``
(``csrc/marshal.c``), because the smallest of these calls take a few microseconds.  Tensors have to lie on the
current device, and a call runs on the current stream unless it is given one; what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import struct
import sys
from array import array

from . import SlopeError, _build, _check, load

EXPORTED_SERVING = ["slope_rope_inv_freq", "slope_qk_norm_rope", "slope_attn_varlen", "slope_kv4_block_bytes",
                    "slope_kv4_cache_bytes", "slope_kv4_write", "slope_kv4_read", "slope_kv4_attn",
                    "slope_kv4_attn_workspace_size"]

ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


class SlopeRope(ctypes.Structure):
    _fields_ = [("begin", ctypes.c_int32), ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("attention_factor", ctypes.c_float), ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class SlopeKV4Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("dqk", ctypes.c_int32), ("dv", ctypes.c_int32)]


def declare(lib):
    """Argument types of the calls of slope_serving.h."""
    P = ctypes.POINTER
    T = ctypes.c_void_p  # a slope_tensor by reference
    i32, i64, vp, f32, f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double
    size = ctypes.c_size_t
    C = ctypes.c_void_p  # a slope_kv4_cache, by reference or as packed bytes
    for name, args, res in (
            ("slope_rope_inv_freq", [i32, f64, ctypes.c_int, f64, f64, f64, f64, P(f64), P(f64)], ctypes.c_int),
            ("slope_qk_norm_rope", [T, T, T, T, ctypes.c_int, f32, vp, vp, i64, T, T, vp], ctypes.c_int),
            ("slope_attn_varlen", [T, T, T, vp, i64, ctypes.c_int, i64, f32, T, T, vp], ctypes.c_int),
            ("slope_kv4_block_bytes", [i32, i32], size),
            ("slope_kv4_cache_bytes", [i64, i32, i32, i32, i32], size),
            ("slope_kv4_write", [C, T, T, vp, vp], ctypes.c_int),
            ("slope_kv4_read", [C, vp, T, T, vp], ctypes.c_int),
            ("slope_kv4_attn", [T, C, vp, i64, i64, vp, i32, i64, f32, T, T, vp, size, vp], ctypes.c_int),
            ("slope_kv4_attn_workspace_size", [i64, i64, C, i32], size)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


_pack_rope = struct.Struct("@iiifP").pack  # slope_rope
_pack_cache = struct.Struct("@Pqiiii").pack  # slope_kv4_cache
_marshal = None  # the C module, once the first call has found it and the library
torch = None  # PyTorch, with the first call: the package can be imported, and the library used, without it
_device = _raw_stream = None  # the current device; its current stream
_alloc = None  # (size, stride, type) -> a tensor on the current device
_modes = _deterministic = None  # dispatch modes that are on; whether deterministic algorithms are asked for


def _module():
    """The C module built for this interpreter."""
    name = f"{__package__}._marshal"
    if name not in sys.modules:
        path = _build.MARSHAL_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"the serving calls' marshalling is not built ({path}); call ring_attention_slope_gb300.build()")
        spec = importlib.util.spec_from_file_location(name, path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        sys.modules[name] = module
    return sys.modules[name]


def _use_torch():
    global torch, _device, _raw_stream, _alloc, _modes, _deterministic
    if torch is not None:
        return
    import torch as t

    try:  # the allocation alone: torch.empty's argument parsing costs a small call another 0.7 us for each output
        from torch._C import _get_deterministic_algorithms as deterministic
        from torch._C import _len_torch_dispatch_stack as modes
        from torch._C._dynamo.guards import _empty_strided_cuda as alloc
    except ImportError:
        alloc, modes, deterministic = _dispatched_alloc, int, bool
    _device, _raw_stream = t._C._cuda_getDevice, t._C._cuda_getCurrentRawStream
    _alloc, _modes, _deterministic = alloc, modes, deterministic
    torch = t


def _dispatched_alloc(size, stride, dtype):
    return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _bound():
    """The C module, bound to the library's calls."""
    global _marshal
    lib = load()
    m = _module()
    _use_torch()
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    m.bind(torch.bfloat16, torch.float32, torch.int32, address(lib.slope_qk_norm_rope), address(lib.slope_attn_varlen),
           address(lib.slope_kv4_write), address(lib.slope_kv4_read), address(lib.slope_kv4_attn),
           address(lib.slope_kv4_cache_bytes), address(lib.slope_kv4_attn_workspace_size))
    _marshal = m
    return m


def _stream(stream, dev):
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _allocator(stream):
    """How a call on the stream allocates.  What it allocates belongs to the stream it runs on: a temporary's memory
    is not handed out again before that stream is done with it.  Where PyTorch's dispatcher has something to do with an
    allocation (a mode watches, or deterministic algorithms have uninitialised memory filled) it goes that way."""
    if stream is None:
        return _dispatched_alloc if _modes() or _deterministic() else _alloc

    def alloc(size, stride, dtype):
        with torch.cuda.stream(stream):
            return _dispatched_alloc(size, stride, dtype)
    return alloc


def _heads(alloc, T, H, d, dtype):
    """A dense [T, H, d]."""
    return alloc((T, H, d), (H * d, d, 1), dtype)


# ---------------------------------------------------------------- positions

def rope_inv_freq(dim, base=10000.0, *, scaling="plain", factor=1.0, original=0.0, fast=0.0, slow=0.0):
    """Rotation frequencies (radians per position) of ``dim`` channels and the attention factor, on the host:
    ``(list of dim / 2 floats, float)``.  ``scaling`` stretches them for long contexts: "linear", "ntk", "bands"
    (by wavelength) or "yarn"; see slope_rope_inv_freq."""
    out = (ctypes.c_double * max(1, int(dim) // 2))()
    factor_out = ctypes.c_double(0.0)
    st = load().slope_rope_inv_freq(int(dim), float(base), ROPE_SCALINGS[scaling], float(factor), float(original),
                                    float(fast), float(slow), out, ctypes.byref(factor_out))
    _check(st, "slope_rope_inv_freq")
    return list(out), factor_out.value


class Rope:
    """Rotation of a head's channels [begin, begin + 2 * len(inv_freq)) by position (slope_rope): ``interleaved``
    pairs channels 2i and 2i + 1, else i and i + half; both cos and sin are multiplied by ``attention_factor``."""

    def __init__(self, inv_freq, *, begin=0, interleaved=False, attention_factor=1.0):
        self._freq = freq = array("d", inv_freq)
        address, n = freq.buffer_info()
        self._c = _pack_rope(begin, 2 * n, 1 if interleaved else 0, attention_factor, address)


def qk_norm_rope(q, k=None, *, norm=True, q_weight=None, k_weight=None, eps=1e-6, rope=None, positions=None, pos0=0,
                 q_out=None, k_out=None, out_dtype=None, stream=None):
    """RMS norm of every head of q [T,Hq,d] and k [T,Hkv,d] and the rotation of its channels by position, one pass.

    Weights: fp32 or bf16, [d] for every head or [H,d].  ``rope``: a :class:`Rope`, or None for the norm alone;
    ``norm=False`` rotates alone.  ``positions``: device int32 [T], or None for pos0, pos0 + 1, ...  The outputs
    (of the inputs' type unless given) may be the inputs.  Returns ``(q_out, k_out)`` (k_out None without k).
    """
    m = _marshal or _bound()
    alloc = _allocator(stream)
    if q_out is None:
        T, H, d = q.shape
        q_out = _heads(alloc, T, H, d, out_dtype or q.dtype)
    if k is not None and k_out is None:
        T, H, d = k.shape
        k_out = _heads(alloc, T, H, d, out_dtype or k.dtype)
    dev = _device()
    st = m.qk_norm_rope(q, k, q_weight, k_weight, norm, eps, None if rope is None else rope._c, positions, pos0, q_out,
                        k_out, _stream(stream, dev), dev)
    _check(st, "slope_qk_norm_rope")
    return q_out, k_out


# ---------------------------------------------------------------- packed prompts

def attn_varlen(q, k, v, cu_seqlens, *, causal=True, window=0, scale=0.0, out=None, lse=None, out_dtype=None,
                stream=None):
    """Attention over prompts packed in q [T,Hq,dqk], k [T,Hkv,dqk], v [T,Hkv,dv] (bf16, CUDA): sequence s is rows
    cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (a host list of ints, or a CPU tensor) and sees only its own keys.

    Returns ``(out, lse)``: out bf16 (default) or fp32 [T,Hq,dv], lse fp32 [Hq,T].  Rows outside the sequences
    are left as they were (uninitialised where the call allocates).
    """
    m = _marshal or _bound()
    alloc = _allocator(stream)
    T, Hq, _ = q.shape
    if out is None:
        out = _heads(alloc, T, Hq, v.shape[2], out_dtype or torch.bfloat16)
    if lse is None:
        lse = alloc((Hq, T), (T, 1), torch.float32)
    if isinstance(cu_seqlens, torch.Tensor):
        if cu_seqlens.is_cuda:
            raise TypeError("cu_seqlens lives on the host (reading it back would synchronise)")
        cu_seqlens = cu_seqlens.tolist()
    dev = _device()
    st = m.attn_varlen(q, k, v, cu_seqlens, causal, window, scale, out, lse, _stream(stream, dev), dev)
    _check(st, "slope_attn_varlen")
    return out, lse


# ---------------------------------------------------------------- the 4-bit cache

class KV4Cache:
    """A paged key/value cache of one layer in 4 bits (slope_kv4_cache): n_pages pages of page_size tokens, Hkv heads
    of dqk key and dv value channels.  ``data`` (uint8, CUDA, dense) is allocated unless given; another tensor may take
    its place later, and a tensor whose memory moves is followed.  The sizes stay as they are."""

    n_pages, page_size, Hkv, dqk, dv = (property(lambda self, i=i: self._sizes[i]) for i in range(5))

    def __init__(self, n_pages, page_size, Hkv, dqk, dv, *, data=None, device="cuda"):
        self._sizes = (n_pages, page_size, Hkv, dqk, dv)
        self._nbytes = nbytes = (_marshal or _bound()).cache_bytes(n_pages, page_size, Hkv, dqk, dv)
        if nbytes == 0 and n_pages != 0:
            raise SlopeError(-8, "slope_kv4_cache_bytes")
        self.data = torch.empty((nbytes,), dtype=torch.uint8, device=device) if data is None else data

    @property
    def data(self):
        return self._data

    @data.setter
    def data(self, data):
        nbytes = self._nbytes
        if data.dtype != torch.uint8 or not data.is_contiguous():
            raise TypeError("the cache's data must be a dense uint8 tensor")
        storage, offset, device = data.untyped_storage(), data.storage_offset(), data.get_device()
        room = min(data.numel(), storage.nbytes() - offset)
        if room < nbytes:
            raise ValueError(f"the cache needs {nbytes} bytes, data holds {room}")
        if nbytes > 0 and device < 0:
            raise TypeError("the cache's data must be a CUDA tensor")
        self._data, self._device, self._address = data, device if nbytes else None, data.data_ptr()
        self._storage, self._end = storage, offset + nbytes  # which has to go on holding as many bytes
        self._c = _pack_cache(self._address if nbytes else 0, *self._sizes)

    def device_now(self):
        """The current device, which the cache's data has to be on, wherever its memory now is."""
        if self._data.data_ptr() != self._address or self._storage.nbytes() < self._end:
            self.data = self._data  # moved or cut short in place: look it over again
        dev = _device()
        if self._device != dev and self._device is not None:
            raise ValueError(f"cache on {self._data.device}, but the current device is cuda:{dev}")
        return dev


def kv4_write(cache, k, v, slots, *, stream=None):
    """Writes k [T,Hkv,dqk], v [T,Hkv,dv] (bf16 or fp32) into the cache at slots (device int32 [T]; slot = page *
    page_size + index, out of range: skipped; the others distinct)."""
    m = _marshal or _bound()
    dev = cache.device_now()
    st = m.kv4_write(cache._c, k, v, slots, _stream(stream, dev), dev)
    _check(st, "slope_kv4_write")


def kv4_read(cache, slots, *, k_out=None, v_out=None, out_dtype=None, stream=None):
    """The values the cache holds at slots (device int32 [T]): ``(k [T,Hkv,dqk], v [T,Hkv,dv])``, bf16 (default) or
    fp32.  Rows whose slot is out of range are left as they were (uninitialised where the call allocates)."""
    m = _marshal or _bound()
    alloc = _allocator(stream)
    T = slots.shape[0]
    if k_out is None:
        k_out = _heads(alloc, T, cache.Hkv, cache.dqk, out_dtype or torch.bfloat16)
    if v_out is None:
        v_out = _heads(alloc, T, cache.Hkv, cache.dv, out_dtype or torch.bfloat16)
    dev = cache.device_now()
    st = m.kv4_read(cache._c, slots, k_out, v_out, _stream(stream, dev), dev)
    _check(st, "slope_kv4_read")
    return k_out, v_out


def kv4_attn_workspace_size(B, Hq, cache, q_len=1) -> int:
    """Workspace bytes of :func:`kv4_attn` (0 for arguments it does not support)."""
    return (_marshal or _bound()).attn_workspace_size(B, Hq, cache._c, q_len)


def kv4_attn(q, cache, block_table, kv_lens, *, q_len=1, window=0, scale=0.0, out=None, lse=None, workspace=None,
             out_dtype=None, want_lse=True, stream=None):
    """Attention of the newest q_len tokens of each sequence, q bf16 [B * q_len,Hq,dqk], over its pages of the cache.

    ``block_table``: device int32 [B,max_pages]; ``kv_lens``: device int32 [B], the newest tokens included.  Token i
    of a sequence sees positions up to kv_lens - q_len + i (and, with ``window``, that many back).  Returns
    ``(out, lse)``: out bf16 (default) or fp32 [B * q_len,Hq,dv], lse fp32 [Hq,B * q_len] (None if not wanted).
    """
    m = _marshal or _bound()
    alloc = _allocator(stream)
    T, Hq, _ = q.shape
    if out is None:
        out = _heads(alloc, T, Hq, cache.dv, out_dtype or torch.bfloat16)
    if lse is None and want_lse:
        lse = alloc((Hq, T), (T, 1), torch.float32)
    if workspace is None:
        nbytes = m.attn_workspace_size(block_table.shape[0], Hq, cache._c, q_len)
        if nbytes == 0:
            raise SlopeError(-8, "slope_kv4_attn_workspace_size")
        workspace = alloc((nbytes,), (1,), torch.uint8)
    elif not workspace.is_contiguous():  # its bytes are counted, and used as one run
        raise ValueError("the workspace must be a dense tensor")
    dev = cache.device_now()
    if workspace.get_device() != dev:
        raise ValueError(f"workspace on {workspace.device}, but the current device is cuda:{dev}")
    st = m.kv4_attn(q, cache._c, block_table, kv_lens, q_len, window, scale, out, lse, workspace.data_ptr(),
                    workspace.nbytes, _stream(stream, dev), dev)
    _check(st, "slope_kv4_attn")
    return out, lse
