"""The 16-bit paged cache (``include/slope_kv.h``): the store, attention of new tokens over its pages, the weights that
the cached tokens got, and eviction by them.

Defaults and outputs are made here; the arguments go to the library through the C module ``_marshal``, as those of the
other serving calls do (:mod:`.serving`).  Tensors have to lie on the current device, and a call runs on the current
stream unless it is given one; what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import struct

from . import SlopeError, _check, load, serving
from .serving import _allocator, _heads, _stream

EXPORTED_KV = ["slope_kv_write", "slope_kv_attn", "slope_kv_attn_workspace_size", "slope_kv_attn_weights",
               "slope_kv_attn_weights_workspace_size", "slope_kv_evict", "slope_kv_evict_workspace_size"]


class SlopeKVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("dqk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3)]


class SlopeKVBatch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("cu_q", ctypes.c_void_p), ("q_len", ctypes.c_int32),
                ("kv_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int64)]


def declare(lib):
    """Argument types of the calls of slope_kv.h."""
    T = C = Bt = ctypes.c_void_p  # a slope_tensor, slope_kv_cache, slope_kv_batch by reference
    i32, i64, vp, f32, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    c_int = ctypes.c_int
    for name, args, res in (
            ("slope_kv_write", [C, T, T, vp, T, vp], c_int),
            ("slope_kv_attn", [T, C, Bt, i64, f32, T, T, vp, size, vp], c_int),
            ("slope_kv_attn_workspace_size", [i64, i64, C, i32], size),
            ("slope_kv_attn_weights", [T, C, Bt, T, i64, f32, c_int, T, vp, size, vp], c_int),
            ("slope_kv_attn_weights_workspace_size", [i64, i64, C, i32], size),
            ("slope_kv_evict", [C, T, i64, vp, i64, i64, vp, i64, i64, i64, vp, i64, i64, vp, vp, vp, size, vp], c_int),
            ("slope_kv_evict_workspace_size", [i64, i64, i64], size)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


_pack_cache = struct.Struct("@PPqiiii6q").pack  # slope_kv_cache
_marshal = None  # the C module, once the first call has found it and the library
torch = None
_device = None


def _bound():
    """The C module, bound to the library's calls on the cache."""
    global _marshal, torch, _device
    m = serving._bound()
    lib = load()
    m.bind_kv(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                for name in ("slope_kv_write", "slope_kv_attn", "slope_kv_attn_weights", "slope_kv_evict",
                             "slope_kv_attn_workspace_size", "slope_kv_attn_weights_workspace_size",
                             "slope_kv_evict_workspace_size")))
    torch, _device = serving.torch, serving._device
    _marshal = m
    return m


class _Pages:
    """One of a cache's two tensors, and where its memory was when last looked at."""

    def __init__(self, t, shape, what):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != shape:
            raise TypeError(f"the cache's {what} must be bf16 {list(shape)}, got {t.dtype} {list(t.shape)}")
        if t.stride(3) != 1:
            raise ValueError(f"the cache's {what} needs contiguous channels")
        self.t = t
        self.look()

    def look(self):
        t = self.t
        self.storage, self.address, self.device = t.untyped_storage(), t.data_ptr(), t.get_device()
        self.end = 2 * (t.storage_offset() + sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1)
        if self.storage.nbytes() < self.end:
            raise ValueError("the cache's memory is smaller than its tensors")
        if self.device < 0:
            raise TypeError("the cache's tensors must be CUDA tensors")

    def moved(self):
        return self.t.data_ptr() != self.address or self.storage.nbytes() < self.end


class KVCache:
    """A paged key/value cache of one layer in bf16 (slope_kv_cache): n_pages pages of page_size tokens, Hkv heads of
    dqk key and dv value channels.  ``k`` [n_pages, Hkv, page_size, dqk] and ``v`` [n_pages, Hkv, page_size, dv] (CUDA)
    are allocated unless given; views of other layouts (token-major pages, say) serve as they are.  A tensor whose
    memory moves is followed."""

    n_pages, page_size, Hkv, dqk, dv = (property(lambda self, i=i: self._sizes[i]) for i in range(5))
    k, v = (property(lambda self, i=i: self._pages[i].t) for i in range(2))

    def __init__(self, n_pages, page_size, Hkv, dqk, dv, *, k=None, v=None, device="cuda"):
        _marshal or _bound()
        self._sizes = (n_pages, page_size, Hkv, dqk, dv)
        shapes = [(n_pages, Hkv, page_size, d) for d in (dqk, dv)]
        k, v = (torch.empty(s, dtype=torch.bfloat16, device=device) if t is None else t for t, s in zip((k, v), shapes))
        self._pages = tuple(_Pages(t, s, what) for t, s, what in zip((k, v), shapes, ("keys", "values")))
        self._look()

    def _look(self):
        a, b = self._pages
        a.look(), b.look()
        # the distance of a single page, head or token is never used
        strides = (s if n > 1 else 8 for p in (a, b) for n, s in zip(p.t.shape[:3], p.t.stride()))
        self._c = _pack_cache(a.address, b.address, *self._sizes, *strides)

    def device_now(self):
        """The current device, which the cache has to be on, wherever its memory now is."""
        a, b = self._pages
        if a.moved() or b.moved():
            self._look()
        dev = _device()
        if a.device != dev or b.device != dev:
            raise ValueError(f"cache on {a.t.device} and {b.t.device}, but the current device is cuda:{dev}")
        return dev


def _workspace(workspace, nbytes, alloc, dev, what):
    """(address, bytes, tensor) of the caller's workspace or of one allocated here."""
    if workspace is None:
        if nbytes == 0:
            raise SlopeError(-8, what)
        workspace = alloc((nbytes,), (1,), torch.uint8)
    elif not workspace.is_contiguous():  # its bytes are counted, and used as one run
        raise ValueError("the workspace must be a dense tensor")
    if workspace.get_device() != dev:
        raise ValueError(f"workspace on {workspace.device}, but the current device is cuda:{dev}")
    return workspace.data_ptr(), workspace.nbytes, workspace


def kv_write(cache, k, v, slots, *, weights=None, stream=None):
    """Writes k [T,Hkv,dqk], v [T,Hkv,dv] (bf16 or fp32) into the cache at slots (device int32 [T]; slot = page *
    page_size + index, out of range: skipped; the others distinct).  With ``weights`` (fp32 [n_pages,Hkv,page_size]) the
    accumulated weights of those slots become 0."""
    m = _marshal or _bound()
    dev = cache.device_now()
    _check(m.kv_write(cache._c, k, v, slots, weights, _stream(stream, dev), dev), "slope_kv_write")


def kv_attn_workspace_size(T, Hq, cache, q_len=0) -> int:
    """Workspace bytes of :func:`kv_attn` for T rows in runs of q_len, or (q_len = 0) in those that a ``cu_q`` gives; 0 for
    arguments it does not support."""
    return (_marshal or _bound()).kv_attn_workspace_size(T, Hq, cache._c, q_len, False)


def kv_attn(q, cache, block_table, kv_lens, *, cu_q=None, q_len=1, window=0, scale=0.0, out=None, lse=None,
            workspace=None, out_dtype=None, want_lse=True, stream=None):
    """Attention of each sequence's newest tokens, rows of q bf16 [T,Hq,dqk], over its pages of the cache.

    The newest tokens of sequence b are rows cu_q[b] .. cu_q[b + 1] - 1 (``cu_q``: device int32 [B + 1]) or, without
    ``cu_q``, rows b * q_len .. (b + 1) * q_len - 1.  ``block_table``: device int32 [B,max_pages]; ``kv_lens``: device
    int32 [B], tokens in the cache, the newest included.  A token sees positions up to its own (and, with ``window``,
    that many back).  Returns ``(out, lse)``: out bf16 (default) or fp32 [T,Hq,dv], lse fp32 [Hq,T] (None if not
    wanted).  Rows of no sequence are left as they were (uninitialised where the call allocates).
    """
    m = _marshal or _bound()
    alloc = _allocator(stream)
    T, Hq, _ = q.shape
    if out is None:
        out = _heads(alloc, T, Hq, cache.dv, out_dtype or torch.bfloat16)
    if lse is None and want_lse:
        lse = alloc((Hq, T), (T, 1), torch.float32)
    dev = cache.device_now()
    nbytes = 0 if workspace is not None else m.kv_attn_workspace_size(T, Hq, cache._c, 0 if cu_q is not None else q_len, False)
    address, nbytes, workspace = _workspace(workspace, nbytes, alloc, dev, "slope_kv_attn_workspace_size")
    st = m.kv_attn(q, cache._c, block_table, kv_lens, cu_q, q_len, window, scale, out, lse, address, nbytes,
                   _stream(stream, dev), dev)
    _check(st, "slope_kv_attn")
    return out, lse


def kv_attn_weights_workspace_size(T, Hq, cache, q_len=0) -> int:
    """Workspace bytes of :func:`kv_attn_weights`, as :func:`kv_attn_workspace_size`."""
    return (_marshal or _bound()).kv_attn_workspace_size(T, Hq, cache._c, q_len, True)


def kv_attn_weights(q, cache, block_table, kv_lens, lse, weights, *, cu_q=None, q_len=1, window=0, scale=0.0,
                    accumulate=True, workspace=None, stream=None):
    """Adds to ``weights`` (fp32 [n_pages,Hkv,page_size]) the attention weight exp(scale q k - lse) that each cached
    token gets from each sequence's newest tokens, summed over them and the query heads of its key head;
    ``accumulate=False`` puts the sums in its place.  ``lse``: fp32 [Hq,T], of :func:`kv_attn` on the same rows (-inf: the
    row adds nothing); the other arguments are as there, but no page may be of two sequences.  Returns ``weights``."""
    m = _marshal or _bound()
    alloc = _allocator(stream)
    T, Hq, _ = q.shape
    dev = cache.device_now()
    nbytes = 0 if workspace is not None else m.kv_attn_workspace_size(T, Hq, cache._c, 0 if cu_q is not None else q_len, True)
    address, nbytes, workspace = _workspace(workspace, nbytes, alloc, dev, "slope_kv_attn_weights_workspace_size")
    st = m.kv_attn_weights(q, cache._c, block_table, kv_lens, cu_q, q_len, lse, window, scale, accumulate, weights,
                           address, nbytes, _stream(stream, dev), dev)
    _check(st, "slope_kv_attn_weights")
    return weights


def kv_evict_workspace_size(B, cache, keep) -> int:
    """Workspace bytes of :func:`kv_evict` (0 for arguments it does not support)."""
    return (_marshal or _bound()).kv_evict_workspace_size(B, cache.Hkv, keep)


def kv_evict(cache, weights, block_table, kv_lens, keep, *, first=0, recent=0, out_table=None, kept=None, out_lens=None,
             workspace=None, stream=None):
    """Keeps of each sequence and key head ``keep`` tokens: the first ``first``, the last ``recent`` and of those between
    the ones with the largest ``weights`` (fp32 [n_pages,Hkv,page_size]; of equal ones the earlier).  They move, in
    order, to the sequence's positions 0, 1, ..., or to those of the pages of ``out_table`` (device int32 [B,pages]);
    weights move along.  The pages that they go to may be no other pages of the call: sequences that share pages need an
    ``out_table``.  Returns ``(kept, out_lens)``: device int32
    [B,Hkv,keep], the kept tokens' old positions and -1 after them, and [B], the new lengths."""
    m = _marshal or _bound()
    alloc = _allocator(stream)
    B, H = kv_lens.shape[0], cache.Hkv
    dev = cache.device_now()
    if kept is None:
        kept = alloc((B, H, keep), (H * keep, keep, 1), torch.int32)
    elif tuple(kept.shape) != (B, H, keep) or not kept.is_contiguous():
        raise ValueError(f"kept must be a dense [{B}, {H}, {keep}], got {list(kept.shape)}")
    if out_lens is None:
        out_lens = alloc((B,), (1,), torch.int32)
    nbytes = 0 if workspace is not None else m.kv_evict_workspace_size(B, H, keep)
    address, nbytes, workspace = _workspace(workspace, nbytes, alloc, dev, "slope_kv_evict_workspace_size")
    st = m.kv_evict(cache._c, weights, block_table, kv_lens, keep, first, recent, out_table, kept, out_lens, address,
                    nbytes, _stream(stream, dev), dev)
    _check(st, "slope_kv_evict")
    return kept, out_lens
