"""Caches of keys and values in 8 or 4 bits, and attention of new tokens over
caches behind a prefix that sequences share, as declared in include/mp3d.h
(which states the formats and the mathematics).  Like the other calls these
only marshal arguments: device tensors in, device tensors out, on the current
stream, with no fallback.

A cache is a tuple: (k, v) of (B, T, H, D) in q's dtype, or, in the formats
"e4m3" and "e2m1", (k_codes, k_scales, v_codes, v_scales), uint8 tensors of
(B, T, H, D) or for e2m1 (B, T, H, (D + 1) // 2), and of
(B, T, H, (D + 31) // 32).  Strides over B, T and H are free; laid out head by
head, as mp3d_cache_empty does, attention reads a head's rows in one piece.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _lib
from .tokens import _code, _contiguous, _heads, _i64x3, _lend, _ptr, _same, _stream

__all__ = ["mp3d_cache_empty", "mp3d_cache_write", "mp3d_cache_read", "mp3d_attention_cached",
           "mp3d_attention_cached_workspace_bytes"]

_FORMAT = {None: _lib.MP3D_CACHE_PLAIN, "e4m3": _lib.MP3D_CACHE_E4M3,
           "e2m1": _lib.MP3D_CACHE_E2M1}
# (packed, as the attention descriptor is: see tokens.py)
_cache_struct = struct.Struct("@qqPPPP12q").pack
_attention_struct = struct.Struct("@iiqqiiii3qff" + 2 * "qqPPPP12q" + "PPiPPPP").pack
_NONE = (0,) * 18
_u8, _i32, _f32 = torch.uint8, torch.int32, torch.float32
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(index, name, *args):
    """Calls the library with the tensors' device as the current one."""
    call = getattr(_lib._lib or _lib.load(), name)
    if index == _current_device():
        code = call(*args)
    else:
        with torch.cuda.device(index):
            code = call(*args)
    if code:
        _lib.check(code)


def _quantised(format):
    code = _FORMAT.get(format, 0)
    if code == 0:
        raise ValueError("format must be 'e4m3' or 'e2m1'")
    return code


def _widths(code, D):
    return D if code == _lib.MP3D_CACHE_E4M3 else (D + 1) // 2, (D + 31) // 32


def _parts(cache, code, D, index, name):
    """The fields of struct mp3d_cache, and H."""
    # (for one new token the calls are bound by the host: nothing here is a
    # call that can be done without)
    if len(cache) == 4:
        kc, ks, vc, vs = cache
        shape, scale = kc.shape, ks.shape
        if len(shape) == 4 and len(scale) == 4 and vc.shape == shape and vs.shape == scale:
            B, T, H, width = shape
            a0, a1, a2, a3 = kc.stride()
            b0, b1, b2, b3 = ks.stride()
            c0, c1, c2, c3 = vc.stride()
            d0, d1, d2, d3 = vs.stride()
            groups = (D + 31) // 32
            if (scale == (B, T, H, groups)
                    and width == (D if code == _lib.MP3D_CACHE_E4M3 else (D + 1) // 2)
                    and kc.dtype is ks.dtype is vc.dtype is vs.dtype is _u8
                    and index == kc.get_device() == ks.get_device() == vc.get_device()
                    == vs.get_device()
                    and (a3 == c3 == 1 or width == 1) and (b3 == d3 == 1 or groups == 1)):
                return (B, T, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), a0, a1,
                        a2, c0, c1, c2, b0, b1, b2, d0, d1, d2), H
    raise ValueError("%s must be (k_codes, k_scales, v_codes, v_scales), uint8 on device %d: codes "
                     "(B, T, H, %d), scales (B, T, H, %d), a head's bytes adjacent"
                     % ((name, index) + _widths(code, D)))


def _per_sequence(t, name, B, index):
    """The address of a (B) int32 tensor, or None."""
    if t is None:
        return None
    if t.shape != (B,) or t.dtype is not _i32 or t.get_device() != index or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape (%d,) on device %d"
                         % (name, B, index))
    return t.data_ptr()


def mp3d_cache_empty(B: int, T: int, H: int, D: int, format: str, device="cuda"):
    """A cache of T rows of H heads of D channels for each of B sequences,
    laid out head by head, its contents not set."""
    width, groups = _widths(_quantised(format), D)
    new = lambda n: torch.empty((B, H, T, n), dtype=torch.uint8,  # noqa: E731
                                device=device).transpose(1, 2)
    return new(width), new(groups), new(width), new(groups)


def mp3d_cache_write(k: torch.Tensor, v: torch.Tensor, cache, format: str, *,
                     start: torch.Tensor | None = None,
                     count: torch.Tensor | None = None) -> None:
    """Quantises k, v (B, T, H, D; any strides over B, T and H) into the cache:
    token t of sequence b to the row start[b] + t.  ``start`` int32 (B) (None:
    0).  ``count`` int32 (B): tokens in use (None: all); those after them,
    and those whose row the cache does not have, are not written."""
    shape, sk = _heads(k, "k")
    vshape, sv = _heads(v, "v", k)
    if vshape != shape:
        raise ValueError("k and v must have the same shape")
    B, T, H, D = shape
    code, index = _quantised(format), k.get_device()
    c, heads = _parts(cache, code, D, index, "cache")
    if c[0] != B or heads != H:
        raise ValueError("the cache must have k's B and H")
    _run(index, "mp3d_cache_write", _cache_struct(*c), code, k.data_ptr(), v.data_ptr(),
         _code(k, "k"), T, H, D, _i64x3(*sk), _i64x3(*sv),
         _per_sequence(start, "start", B, index), _per_sequence(count, "count", B, index),
         _stream(k))


def mp3d_cache_read(cache, format: str, D: int, dtype: torch.dtype, *, rows: int | None = None,
                    start: torch.Tensor | None = None, count: torch.Tensor | None = None,
                    out=None):
    """(k, v) of (B, rows, H, D): the values of the cache's rows start[b] + t
    (``rows`` None: as many as it has; ``start`` None: from 0), zeros from
    count[b] on and where the cache has no such row.  ``out``: preallocated
    contiguous (k, v)."""
    code, first = _quantised(format), cache[0]
    if not first.is_cuda:
        raise ValueError("cache must be device tensors")
    index = first.get_device()
    c, H = _parts(cache, code, D, index, "cache")
    B = c[0]
    T = c[1] if rows is None else rows
    if out is None:
        k = first.new_empty((B, T, H, D), dtype=dtype)
        v = torch.empty_like(k)
    else:
        k, v = out
        _same(k, "out for k", (B, T, H, D), dtype, first.device)
        _same(v, "out for v", (B, T, H, D), dtype, first.device)
    _run(index, "mp3d_cache_read", _cache_struct(*c), code, k.data_ptr(), v.data_ptr(),
         _code(k, "out"), T, H, D, _per_sequence(start, "start", B, index),
         _per_sequence(count, "count", B, index), _stream(k))
    return k, v


def _fields(cache, code, q, name):
    """The fields of struct mp3d_cache of any format, and H."""
    D = q.shape[3]
    if code:
        return _parts(cache, code, D, q.get_device(), name)
    if len(cache) != 2:
        raise ValueError("%s must be (k, v)" % name)
    k, v = cache
    shape, ks = _heads(k, name, q)
    vshape, vs = _heads(v, name, q)
    if vshape != shape or shape[3] != D:
        raise ValueError("%s: k and v must have the shape (B, T, H, %d)" % (name, D))
    return (shape[0], shape[1], k.data_ptr(), v.data_ptr(), 0, 0, *ks, *vs, *(0,) * 6), shape[2]


def _descriptor(q, own, prefix, format, scale, softcap, causal, kv_len, prefix_len, slopes, pos_q,
                pos_k, pos_prefix):
    """struct mp3d_attention_cache, packed."""
    (B, Tq, Hq, D), qs = _heads(q, "q")
    if format not in _FORMAT:
        raise ValueError("format must be 'e4m3', 'e2m1' or None")
    code, dev, index = _FORMAT[format], q.device, q.get_device()
    o, Hk = _fields(own, code, q, "own")
    if o[0] != B:
        raise ValueError("the own cache must have q's B")
    p, N = _NONE, 0
    if prefix is not None:
        p, heads = _fields(prefix, code, q, "prefix")
        N = p[0]
        if heads != Hk:
            raise ValueError("own and prefix must have the same heads")
        if N < 1 or B % N:
            raise ValueError("%d sequences do not divide among %d prefixes" % (B, N))
    axes = psl = ppq = ppk = ppp = 0
    if prefix_len is not None and prefix is None:
        raise ValueError("prefix_len goes with prefix")
    kv = _per_sequence(kv_len, "kv_len", B, index) or 0
    pl = _per_sequence(prefix_len, "prefix_len", N, index) or 0
    if slopes is not None:
        if slopes.dim() != 2 or pos_q is None or pos_k is None or (
                (pos_prefix is None) != (prefix is None)):
            raise ValueError("a distance bias needs slopes (Hq, axes), pos_q, pos_k and, with a "
                             "prefix, pos_prefix")
        axes = slopes.shape[1]
        if not 1 <= axes <= 3:
            raise ValueError("slopes must have 1 to 3 axes")
        psl = _same(slopes, "slopes", (Hq, axes), torch.float32, dev).data_ptr()
        ppq = _same(pos_q, "pos_q", (axes, B, Tq), torch.int32, dev).data_ptr()
        ppk = _same(pos_k, "pos_k", (axes, B, o[1]), torch.int32, dev).data_ptr()
        if prefix is not None:
            ppp = _same(pos_prefix, "pos_prefix", (axes, N, p[1]), torch.int32, dev).data_ptr()
    elif pos_q is not None or pos_k is not None or pos_prefix is not None:
        raise ValueError("positions go with slopes")
    return _attention_struct(_code(q, "q"), code, B, Tq, Hq, Hk, D, 1 if causal else 0, *qs,
                             1.0 / math.sqrt(D) if scale is None and D else float(scale or 0.0),
                             softcap, *o, *p, kv, pl, axes, psl, ppq, ppk, ppp)


def mp3d_attention_cached_workspace_bytes(q, own, prefix=None, *, format=None, scale=None,
                                          softcap=0.0, causal=True, kv_len=None, prefix_len=None,
                                          slopes=None, pos_q=None, pos_k=None,
                                          pos_prefix=None) -> int:
    """Workspace bytes of mp3d_attention_cached with these arguments."""
    a = _descriptor(q, own, prefix, format, scale, softcap, causal, kv_len, prefix_len, slopes,
                    pos_q, pos_k, pos_prefix)
    nbytes = ctypes.c_size_t()
    _run(q.get_device(), "mp3d_attention_cached_workspace_bytes", a, ctypes.byref(nbytes))
    return nbytes.value


def mp3d_attention_cached(q: torch.Tensor, own, prefix=None, *, format: str | None = None,
                          scale=None, softcap: float = 0.0, causal: bool = True,
                          kv_len: torch.Tensor | None = None,
                          prefix_len: torch.Tensor | None = None,
                          slopes: torch.Tensor | None = None, pos_q: torch.Tensor | None = None,
                          pos_k: torch.Tensor | None = None,
                          pos_prefix: torch.Tensor | None = None, out=None,
                          workspace: torch.Tensor | None = None):
    """Attention of new tokens q (B, Tq, Hq, D) over their sequences' caches
    ``own`` (a cache of B sequences, with the new tokens already in it) behind
    ``prefix`` (a cache of N sequences, each shared by B / N sequences that
    follow each other, and read once for them): (out, lse), out
    (B, Tq, Hq, D) and lse float32 (B, Hq, Tq).

    ``format`` "e4m3", "e2m1" or None (plain caches).  ``kv_len`` int32 (B):
    rows of the own caches in use, the new tokens' the last Tq of them
    (``causal``: a token sees those up to its own); ``prefix_len`` int32 (N).
    ``scale``, ``softcap``, ``slopes`` as for mp3d_attention_forward, with
    ``pos_q`` (axes, B, Tq), ``pos_k`` (axes, B, T) and ``pos_prefix``
    (axes, N, P) int32.  ``out``: preallocated (out, lse); ``workspace``: a
    uint8 tensor of mp3d_attention_cached_workspace_bytes(...) (None:
    allocated).

    Over plain caches without a prefix mp3d_attention_forward(kv_len=...)
    gives the same, and has a backward; this is the faster of the two for new
    tokens."""
    a = _descriptor(q, own, prefix, format, scale, softcap, causal, kv_len, prefix_len, slopes,
                    pos_q, pos_k, pos_prefix)
    B, Tq, Hq, _ = shape = q.shape
    index = q.get_device()
    if out is None:
        o = torch.empty_like(q, memory_format=_contiguous)
        lse = q.new_empty((B, Hq, Tq), dtype=_f32)
    else:
        o, lse = out
        _same(o, "out", shape, q.dtype, q.device)
        _same(lse, "lse", (B, Hq, Tq), _f32, q.device)
    nbytes = ctypes.c_size_t()
    _run(index, "mp3d_attention_cached_workspace_bytes", a, ctypes.byref(nbytes))
    ws, n = _lend(nbytes.value, workspace, q.device)
    _run(index, "mp3d_attention_cached", a, q.data_ptr(), o.data_ptr(), lse.data_ptr(), _ptr(ws), n,
         _stream(q))
    return o, lse
