"""The calls around the prefill attention (``include/slope_serving.h``): head norm with rotation, packed
prompts, the 4-bit paged key/value cache and attention over it.

Argument marshalling only, as in the package's ``__init__``: tensors have to lie on the current device, and a
call runs on the current stream unless it is given one.
"""
from __future__ import annotations

import ctypes

from . import SlopeError, SlopeTensor, _check, _desc, _stream_ptr, _torch, load

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
    T = P(SlopeTensor)
    i32, i64, vp, f32, f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double
    size = ctypes.c_size_t
    C = P(SlopeKV4Cache)
    for name, args, res in (
            ("slope_rope_inv_freq", [i32, f64, ctypes.c_int, f64, f64, f64, f64, P(f64), P(f64)], ctypes.c_int),
            ("slope_qk_norm_rope", [T, T, T, T, ctypes.c_int, f32, P(SlopeRope), vp, i64, T, T, vp], ctypes.c_int),
            ("slope_attn_varlen", [T, T, T, P(i64), i64, ctypes.c_int, i64, f32, T, T, vp], ctypes.c_int),
            ("slope_kv4_block_bytes", [i32, i32], size),
            ("slope_kv4_cache_bytes", [i64, i32, i32, i32, i32], size),
            ("slope_kv4_write", [C, T, T, vp, vp], ctypes.c_int),
            ("slope_kv4_read", [C, vp, T, T, vp], ctypes.c_int),
            ("slope_kv4_attn", [T, C, vp, i64, i64, vp, i32, i64, f32, T, T, vp, size, vp], ctypes.c_int),
            ("slope_kv4_attn_workspace_size", [i64, i64, C, i32], size)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


def _ref(d):
    return ctypes.byref(d) if d is not None else None


def _here(*tensors):
    """The tensors' device has to be the current one: the launch goes to the current device's stream."""
    torch = _torch()
    for t in tensors:
        if t is not None and t.is_cuda and t.device.index != torch.cuda.current_device():
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _index(t, what, n=None):
    """Data pointer of a device int32 array (dense, of n elements)."""
    torch = _torch()
    if t.dtype != torch.int32:
        raise TypeError(f"{what} must be int32, got {t.dtype}")
    if t.numel() > 0 and t.device.type != "cuda":
        raise TypeError(f"{what} must be a CUDA tensor")
    if n is not None and (t.dim() != 1 or t.shape[0] != n):
        raise ValueError(f"{what} must have shape [{n}], got {tuple(t.shape)}")
    if t.dim() == 1 and t.numel() > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")
    return ctypes.c_void_p(t.data_ptr() if t.numel() > 0 else 0)


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
        self._freq = (ctypes.c_double * max(1, len(inv_freq)))(*[float(f) for f in inv_freq])
        self._c = SlopeRope(int(begin), 2 * len(inv_freq), int(bool(interleaved)), float(attention_factor),
                            ctypes.cast(self._freq, ctypes.POINTER(ctypes.c_double)))


def qk_norm_rope(q, k=None, *, norm=True, q_weight=None, k_weight=None, eps=1e-6, rope=None, positions=None, pos0=0,
                 q_out=None, k_out=None, out_dtype=None, stream=None):
    """RMS norm of every head of q [T,Hq,d] and k [T,Hkv,d] and the rotation of its channels by position, one pass.

    Weights: fp32 or bf16, [d] for every head or [H,d].  ``rope``: a :class:`Rope`, or None for the norm alone;
    ``norm=False`` rotates alone.  ``positions``: device int32 [T], or None for pos0, pos0 + 1, ...  The outputs
    (of the inputs' type unless given) may be the inputs.  Returns ``(q_out, k_out)`` (k_out None without k).
    """
    torch = _torch()
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    if k is not None and k_out is None:
        k_out = torch.empty(k.shape, dtype=out_dtype or k.dtype, device=k.device)
    _here(q, k, q_weight, k_weight, positions, q_out, k_out)
    weights = [None if w is None else _desc(w.unsqueeze(0) if w.dim() == 1 else w) for w in (q_weight, k_weight)]
    pos = None if positions is None else _index(positions, "positions", q.shape[0])
    dq, do = _desc(q), _desc(q_out)
    dk, dko = (_desc(k), _desc(k_out)) if k is not None else (None, None)
    st = load().slope_qk_norm_rope(_ref(dq), _ref(dk), _ref(weights[0]), _ref(weights[1]), int(bool(norm)), float(eps),
                                   _ref(rope._c) if rope is not None else None, pos, int(pos0), _ref(do), _ref(dko),
                                   _stream_ptr(stream))
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
    torch = _torch()
    T, Hq, _ = q.shape
    if out is None:
        out = torch.empty((T, Hq, v.shape[2]), dtype=out_dtype or torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    _here(q, k, v, out, lse)
    if hasattr(cu_seqlens, "tolist"):
        if getattr(cu_seqlens, "is_cuda", False):
            raise TypeError("cu_seqlens lives on the host (reading it back would synchronise)")
        cu_seqlens = cu_seqlens.tolist()
    if len(cu_seqlens) < 1:
        raise ValueError("cu_seqlens needs at least one entry")
    cu = (ctypes.c_int64 * len(cu_seqlens))(*[int(c) for c in cu_seqlens])
    dq, dk, dvv, do, dl = _desc(q), _desc(k), _desc(v), _desc(out), _desc(lse)
    st = load().slope_attn_varlen(_ref(dq), _ref(dk), _ref(dvv), cu, len(cu_seqlens) - 1, int(bool(causal)),
                                  int(window), float(scale), _ref(do), _ref(dl), _stream_ptr(stream))
    _check(st, "slope_attn_varlen")
    return out, lse


# ---------------------------------------------------------------- the 4-bit cache

class KV4Cache:
    """A paged key/value cache of one layer in 4 bits (slope_kv4_cache): n_pages pages of page_size tokens, Hkv heads
    of dqk key and dv value channels.  ``data`` (uint8, CUDA, dense) is allocated unless given."""

    def __init__(self, n_pages, page_size, Hkv, dqk, dv, *, data=None, device="cuda"):
        torch = _torch()
        nbytes = int(load().slope_kv4_cache_bytes(int(n_pages), int(page_size), int(Hkv), int(dqk), int(dv)))
        if nbytes == 0 and int(n_pages) != 0:
            raise SlopeError(-8, "slope_kv4_cache_bytes")
        if data is None:
            data = torch.empty((nbytes,), dtype=torch.uint8, device=device)
        if data.dtype != torch.uint8 or not data.is_contiguous():
            raise TypeError("the cache's data must be a dense uint8 tensor")
        if nbytes > 0 and data.device.type != "cuda":
            raise TypeError("the cache's data must be a CUDA tensor")
        if data.numel() < nbytes:
            raise ValueError(f"the cache needs {nbytes} bytes, data holds {data.numel()}")
        self.data = data
        self.n_pages, self.page_size, self.Hkv, self.dqk, self.dv = (int(x) for x in (n_pages, page_size, Hkv, dqk, dv))
        self._c = SlopeKV4Cache(data.data_ptr() if nbytes else None, self.n_pages, self.page_size, self.Hkv, self.dqk,
                                self.dv)


def kv4_write(cache, k, v, slots, *, stream=None):
    """Writes k [T,Hkv,dqk], v [T,Hkv,dv] (bf16 or fp32) into the cache at slots (device int32 [T]; slot = page *
    page_size + index, out of range: skipped; the others distinct)."""
    _here(cache.data, k, v, slots)
    dk, dv = _desc(k), _desc(v)
    st = load().slope_kv4_write(_ref(cache._c), _ref(dk), _ref(dv), _index(slots, "slots", k.shape[0]),
                                _stream_ptr(stream))
    _check(st, "slope_kv4_write")


def kv4_read(cache, slots, *, k_out=None, v_out=None, out_dtype=None, stream=None):
    """The values the cache holds at slots (device int32 [T]): ``(k [T,Hkv,dqk], v [T,Hkv,dv])``, bf16 (default) or
    fp32.  Rows whose slot is out of range are left as they were (uninitialised where the call allocates)."""
    torch = _torch()
    T = slots.shape[0]
    if k_out is None:
        k_out = torch.empty((T, cache.Hkv, cache.dqk), dtype=out_dtype or torch.bfloat16, device=cache.data.device)
    if v_out is None:
        v_out = torch.empty((T, cache.Hkv, cache.dv), dtype=out_dtype or torch.bfloat16, device=cache.data.device)
    _here(cache.data, slots, k_out, v_out)
    dk, dv = _desc(k_out), _desc(v_out)
    st = load().slope_kv4_read(_ref(cache._c), _index(slots, "slots", k_out.shape[0]), _ref(dk), _ref(dv),
                               _stream_ptr(stream))
    _check(st, "slope_kv4_read")
    return k_out, v_out


def kv4_attn_workspace_size(B, Hq, cache, q_len=1) -> int:
    """Workspace bytes of :func:`kv4_attn` (0 for arguments it does not support)."""
    return int(load().slope_kv4_attn_workspace_size(int(B), int(Hq), _ref(cache._c), int(q_len)))


def kv4_attn(q, cache, block_table, kv_lens, *, q_len=1, window=0, scale=0.0, out=None, lse=None, workspace=None,
             out_dtype=None, want_lse=True, stream=None):
    """Attention of the newest q_len tokens of each sequence, q bf16 [B * q_len,Hq,dqk], over its pages of the cache.

    ``block_table``: device int32 [B,max_pages]; ``kv_lens``: device int32 [B], the newest tokens included.  Token i
    of a sequence sees positions up to kv_lens - q_len + i (and, with ``window``, that many back).  Returns
    ``(out, lse)``: out bf16 (default) or fp32 [B * q_len,Hq,dv], lse fp32 [Hq,B * q_len] (None if not wanted).
    """
    torch = _torch()
    T, Hq, _ = q.shape
    if out is None:
        out = torch.empty((T, Hq, cache.dv), dtype=out_dtype or torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    q_len = int(q_len)
    if q_len < 1 or T % q_len != 0:
        raise ValueError(f"q has {T} rows, not a multiple of q_len = {q_len}")
    B = T // q_len
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must have shape [{B}, pages], got {tuple(block_table.shape)}")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    if workspace is None:
        nbytes = kv4_attn_workspace_size(B, Hq, cache, q_len)
        if nbytes == 0:
            raise SlopeError(-8, "slope_kv4_attn_workspace_size")
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=q.device)
    _here(q, cache.data, block_table, kv_lens, out, lse, workspace)
    dq, do = _desc(q), _desc(out)
    dl = _desc(lse) if lse is not None else None
    st = load().slope_kv4_attn(_ref(dq), _ref(cache._c), _index(block_table, "block_table"),
                               block_table.stride(0) if B > 1 else block_table.shape[1], block_table.shape[1],
                               _index(kv_lens, "kv_lens", B), q_len, int(window), float(scale), _ref(do), _ref(dl),
                               ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
                               _stream_ptr(stream))
    _check(st, "slope_kv4_attn")
    return out, lse
