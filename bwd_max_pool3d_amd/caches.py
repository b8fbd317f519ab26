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


def _on(device, call, *args):
    """The call's result, with the tensors' device as the current one."""
    if device.index == torch.cuda.current_device():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _quantised(format):
    code = _FORMAT.get(format, 0)
    if code == 0:
        raise ValueError("format must be 'e4m3' or 'e2m1'")
    return code


def _widths(code, D):
    return D if code == _lib.MP3D_CACHE_E4M3 else (D + 1) // 2, (D + 31) // 32


def _bytes(t, name, device):
    """(shape, first three strides) of a part of a cache."""
    shape, strides = t.shape, t.stride()
    if t.dtype != torch.uint8 or len(shape) != 4 or t.device != device:
        raise ValueError("%s must be a uint8 tensor (B, T, H, bytes) on %s" % (name, device))
    if strides[3] != 1 and shape[3] > 1:
        raise ValueError("%s: a head's bytes must be adjacent (stride 1)" % name)
    return shape, strides[:3]


def _parts(cache, code, D, device, name):
    """The fields of struct mp3d_cache, and H."""
    if len(cache) != 4:
        raise ValueError("%s must be (k_codes, k_scales, v_codes, v_scales)" % name)
    kc, ks, vc, vs = cache
    shape, s0 = _bytes(kc, name, device)
    scale, s1 = _bytes(ks, name, device)
    vshape, s2 = _bytes(vc, name, device)
    vscale, s3 = _bytes(vs, name, device)
    B, T, H, width = shape
    if (vshape != shape or vscale != scale or scale[:3] != shape[:3]
            or (width, scale[3]) != _widths(code, D)):
        raise ValueError("%s must have codes (B, T, H, %d) and scales (B, T, H, %d)"
                         % ((name,) + _widths(code, D)))
    return (B, T, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), *s0, *s2, *s1,
            *s3), H


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
    lib = _lib.load()
    shape, sk = _heads(k, "k")
    vshape, sv = _heads(v, "v", k)
    if vshape != shape:
        raise ValueError("k and v must have the same shape")
    B, T, H, D = shape
    code, dev = _quantised(format), k.device
    c, heads = _parts(cache, code, D, dev, "cache")
    if c[0] != B or heads != H:
        raise ValueError("the cache must have k's B and H")
    if start is not None:
        _same(start, "start", (B,), torch.int32, dev)
    if count is not None:
        _same(count, "count", (B,), torch.int32, dev)
    _lib.check(_on(dev, lib.mp3d_cache_write, _cache_struct(*c), code, k.data_ptr(), v.data_ptr(),
                   _code(k, "k"), T, H, D, _i64x3(*sk), _i64x3(*sv), _ptr(start), _ptr(count),
                   _stream(k)))


def mp3d_cache_read(cache, format: str, D: int, dtype: torch.dtype, *, rows: int | None = None,
                    start: torch.Tensor | None = None, count: torch.Tensor | None = None,
                    out=None):
    """(k, v) of (B, rows, H, D): the values of the cache's rows start[b] + t
    (``rows`` None: as many as it has; ``start`` None: from 0), zeros from
    count[b] on and where the cache has no such row.  ``out``: preallocated
    contiguous (k, v)."""
    lib = _lib.load()
    code = _quantised(format)
    if not cache[0].is_cuda:
        raise ValueError("cache must be device tensors")
    dev = cache[0].device
    c, H = _parts(cache, code, D, dev, "cache")
    B = c[0]
    T = c[1] if rows is None else rows
    if out is None:
        k = torch.empty((B, T, H, D), dtype=dtype, device=dev)
        v = torch.empty_like(k)
    else:
        k, v = out
        _same(k, "out for k", (B, T, H, D), dtype, dev)
        _same(v, "out for v", (B, T, H, D), dtype, dev)
    if start is not None:
        _same(start, "start", (B,), torch.int32, dev)
    if count is not None:
        _same(count, "count", (B,), torch.int32, dev)
    _lib.check(_on(dev, lib.mp3d_cache_read, _cache_struct(*c), code, k.data_ptr(), v.data_ptr(),
                   _code(k, "out"), T, H, D, _ptr(start), _ptr(count), _stream(k)))
    return k, v


def _fields(cache, code, q, name):
    """The fields of struct mp3d_cache of any format, and H."""
    D = q.shape[3]
    if code:
        return _parts(cache, code, D, q.device, name)
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
    code, dev = _FORMAT[format], q.device
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
    kv = pl = axes = psl = ppq = ppk = ppp = 0
    if kv_len is not None:
        kv = _same(kv_len, "kv_len", (B,), torch.int32, dev).data_ptr()
    if prefix_len is not None:
        if prefix is None:
            raise ValueError("prefix_len goes with prefix")
        pl = _same(prefix_len, "prefix_len", (N,), torch.int32, dev).data_ptr()
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
    _lib.check(_on(q.device, _lib.load().mp3d_attention_cached_workspace_bytes, a,
                   ctypes.byref(nbytes)))
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
    allocated)."""
    lib = _lib.load()
    a = _descriptor(q, own, prefix, format, scale, softcap, causal, kv_len, prefix_len, slopes,
                    pos_q, pos_k, pos_prefix)
    B, Tq, Hq, _ = q.shape
    dev = q.device
    if out is None:
        o = torch.empty_like(q, memory_format=_contiguous)
        lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=dev)
    else:
        o, lse = out
        _same(o, "out", q.shape, q.dtype, dev)
        _same(lse, "lse", (B, Hq, Tq), torch.float32, dev)
    nbytes = ctypes.c_size_t()
    _lib.check(_on(dev, lib.mp3d_attention_cached_workspace_bytes, a, ctypes.byref(nbytes)))
    ws, n = _lend(nbytes.value, workspace, dev)
    _lib.check(_on(dev, lib.mp3d_attention_cached, a, q.data_ptr(), o.data_ptr(), lse.data_ptr(),
                   _ptr(ws), n, _stream(q)))
    return o, lse
