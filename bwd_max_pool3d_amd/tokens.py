"""Operators over a pooled volume's tokens: rotary positions, attention and
the gated norm, as declared in include/mp3d.h (which states their
mathematics).  Like the pooling calls these only marshal arguments: device
tensors in, device tensors out, on the current stream, with no fallback.

float32, float16 and bfloat16.  q, k, v and their gradients are
(B, T, H, D) with any strides over B, T and H (a cache laid out (B, H, T, D)
is passed as its transpose); a head's channels are adjacent.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _lib

__all__ = ["mp3d_rope_forward", "mp3d_rope_backward", "mp3d_attention_forward",
           "mp3d_attention_backward", "mp3d_attention_workspace_bytes",
           "mp3d_gated_norm_forward", "mp3d_gated_norm_backward",
           "mp3d_gated_norm_workspace_bytes"]

_DTYPE = {torch.float32: _lib.MP3D_F32, torch.float16: _lib.MP3D_F16,
          torch.bfloat16: _lib.MP3D_BF16}
_NORM = {"rms": _lib.MP3D_NORM_RMS, "layer": _lib.MP3D_NORM_LAYER}
# Host arrays and the attention descriptor go to the library as packed bytes:
# for one token the calls are bound by the host, and ctypes arrays and
# structure fields cost several times as much.
_i64x3 = struct.Struct("=qqq").pack
_i32x3 = struct.Struct("=iii").pack
_attention_struct = struct.Struct("@iqqqiii9qffiPPiPiPPP").pack
_contiguous = torch.contiguous_format
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _code(t: torch.Tensor, name: str) -> int:
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise TypeError("%s: unsupported dtype %s" % (name, t.dtype)) from None


def _stream(t: torch.Tensor) -> int:
    """The current stream of t's device, as a hipStream_t."""
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _heads(t: torch.Tensor, name: str, like: torch.Tensor | None = None):
    """(shape, first three strides) of a (B, T, H, D) device tensor with
    adjacent channels."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    shape, strides = t.shape, t.stride()
    if len(shape) != 4:
        raise ValueError("%s must be 4-D (B, T, H, D)" % name)
    if strides[3] != 1 and shape[3] > 1:
        raise ValueError("%s: a head's channels must be adjacent (stride 1)" % name)
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError("%s must have the dtype and device of the first tensor" % name)
    return shape, strides[:3]


def _same(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    """A contiguous device tensor of this shape and dtype."""
    if (t.shape != shape or t.dtype != dtype or t.device != device
            or not t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, tuple(shape), device))
    return t


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()



# ------------------------------------------------------------ rotary positions

def _rope(name, q, k, inv_freq, pairs, positions, grid, interleaved, out):
    lib = _lib.load()
    (B, T, Hq, D), qs = _heads(q, "q")
    code, dev = _code(q, "q"), q.device
    Hk, ks = 0, None
    if k is not None:
        (Bk, T2, Hk, Dk), ks = _heads(k, "k", q)
        if (Bk, T2, Dk) != (B, T, D):
            raise ValueError("q and k must share B, T and D")
    if len(pairs) != 3:
        raise ValueError("pairs must be three counts, one for each axis")
    _same(inv_freq, "inv_freq", (sum(pairs),), torch.float32, dev)
    if (positions is None) == (grid is None):
        raise ValueError("give either positions or grid")
    if positions is not None:
        _same(positions, "positions", (3, B, T), torch.int32, dev)
    elif len(grid) != 3:
        raise ValueError("grid must be three extents (D, H, W)")
    if out is None:
        qo = torch.empty_like(q, memory_format=_contiguous)
        ko = None if k is None else torch.empty_like(k, memory_format=_contiguous)
        row = T * Hq * D, Hq * D, D
        qos, kos = _i64x3(*row), _i64x3(T * Hk * D, Hk * D, D)
    else:
        qo, ko = out if k is not None else (out, None)
        shape, st = _heads(qo, "out for q", q)
        qos = _i64x3(*st)
        if shape != q.shape:
            raise ValueError("out for q must have its input's shape")
        kos = None
        if k is not None:
            shape, st = _heads(ko, "out for k", q)
            kos = _i64x3(*st)
            if shape != k.shape:
                raise ValueError("out for k must have its input's shape")
    _lib.check(getattr(lib, name)(
        q.data_ptr(), _ptr(k), qo.data_ptr(), _ptr(ko), code, B, T, Hq, Hk, D, _i64x3(*qs),
        None if k is None else _i64x3(*ks), qos, kos, inv_freq.data_ptr(), _i32x3(*pairs),
        _ptr(positions), None if grid is None else _i32x3(*grid), 1 if interleaved else 0,
        _stream(q)))
    return qo if k is None else (qo, ko)


def mp3d_rope_forward(q: torch.Tensor, k: torch.Tensor | None, inv_freq: torch.Tensor, pairs,
                      positions: torch.Tensor | None = None, grid=None,
                      interleaved: bool = False, out=None):
    """Rotary positions over three axes: (q', k'), or q' when ``k`` is None.

    ``pairs`` = (pd, ph, pw): how many channel pairs turn by each axis;
    ``inv_freq`` float32 (pd + ph + pw).  Positions are ``positions`` int32
    (3, B, T), or ``grid`` = (D, H, W) for tokens in the scan order of a
    pooled volume.  ``interleaved``: a pair is channels (2i, 2i + 1) rather
    than (i, P + i).  ``out``: preallocated (q', k') (or q'), which may be the
    inputs themselves."""
    return _rope("mp3d_rope_forward", q, k, inv_freq, pairs, positions, grid, interleaved, out)


def mp3d_rope_backward(gq: torch.Tensor, gk: torch.Tensor | None, inv_freq: torch.Tensor, pairs,
                       positions: torch.Tensor | None = None, grid=None,
                       interleaved: bool = False, out=None):
    """Gradients of q and k from those of the turned q' and k'; arguments as
    for mp3d_rope_forward."""
    return _rope("mp3d_rope_backward", gq, gk, inv_freq, pairs, positions, grid, interleaved, out)


# ------------------------------------------------------------------- attention

def _attention(q, k, v, scale, softcap, causal, kv_len, doc_offsets, prefix, slopes, pos_q, pos_k):
    """The call's descriptor (include/mp3d.h, struct mp3d_attention), packed."""
    (B, Tq, Hq, D), qs = _heads(q, "q")
    kshape, ks = _heads(k, "k", q)
    vshape, vs = _heads(v, "v", q)
    Tk, Hk = kshape[1], kshape[2]
    if vshape != kshape or kshape[0] != B or kshape[3] != D:
        raise ValueError("k and v must have the shape (B, Tk, Hk, D) with q's B and D")
    dev = q.device
    kv = docs = pre = 0
    n_docs = axes = psl = ppq = ppk = 0
    if kv_len is not None:
        kv = _same(kv_len, "kv_len", (B,), torch.int32, dev).data_ptr()
    if doc_offsets is not None:
        if doc_offsets.dim() != 2 or doc_offsets.shape[1] < 2:
            raise ValueError("doc_offsets must be (B, n_docs + 1)")
        n_docs = doc_offsets.shape[1] - 1
        docs = _same(doc_offsets, "doc_offsets", (B, n_docs + 1), torch.int32, dev).data_ptr()
    if prefix is not None:
        if prefix.dim() == 1:
            prefix = prefix[:, None]
        pre = _same(prefix, "prefix", (B, n_docs or 1), torch.int32, dev).data_ptr()
    if slopes is not None:
        if slopes.dim() != 2 or pos_q is None or pos_k is None:
            raise ValueError("a distance bias needs slopes (Hq, axes), pos_q and pos_k")
        axes = slopes.shape[1]
        if not 1 <= axes <= 3:
            raise ValueError("slopes must have 1 to 3 axes")
        psl = _same(slopes, "slopes", (Hq, axes), torch.float32, dev).data_ptr()
        ppq = _same(pos_q, "pos_q", (axes, B, Tq), torch.int32, dev).data_ptr()
        ppk = _same(pos_k, "pos_k", (axes, B, Tk), torch.int32, dev).data_ptr()
    elif pos_q is not None or pos_k is not None:
        raise ValueError("pos_q and pos_k go with slopes")
    return _attention_struct(_code(q, "q"), B, Tq, Tk, Hq, Hk, D, *qs, *ks, *vs,
                             1.0 / math.sqrt(D) if scale is None and D else float(scale or 0.0),
                             softcap, 1 if causal else 0, kv, docs, n_docs, pre, axes, psl, ppq,
                             ppk)


def _workspace(lib, a, backward, workspace, device):
    nbytes = ctypes.c_size_t()
    _lib.check(lib.mp3d_attention_workspace_bytes(a, backward, ctypes.byref(nbytes)))
    return _lend(nbytes.value, workspace, device)


def _lend(need, workspace, device):
    """(tensor or None, its bytes): the caller's workspace, or a new one."""
    if workspace is None:
        if need == 0:
            return None, 0
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
            or workspace.device != device):
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    return workspace, workspace.numel()


def mp3d_attention_workspace_bytes(q, k, v, backward: bool = False, *, scale=None, softcap=0.0,
                                   causal=False, kv_len=None, doc_offsets=None, prefix=None,
                                   slopes=None, pos_q=None, pos_k=None) -> int:
    """Workspace bytes of the forward or the backward of these arguments."""
    a = _attention(q, k, v, scale, softcap, causal, kv_len, doc_offsets, prefix, slopes, pos_q,
                   pos_k)
    nbytes = ctypes.c_size_t()
    _lib.check(_lib.load().mp3d_attention_workspace_bytes(a, int(backward),
                                                          ctypes.byref(nbytes)))
    return nbytes.value


def mp3d_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale=None,
                           softcap: float = 0.0, causal: bool = False,
                           kv_len: torch.Tensor | None = None,
                           doc_offsets: torch.Tensor | None = None,
                           prefix: torch.Tensor | None = None,
                           slopes: torch.Tensor | None = None,
                           pos_q: torch.Tensor | None = None, pos_k: torch.Tensor | None = None,
                           out=None, workspace: torch.Tensor | None = None):
    """Attention of q (B, Tq, Hq, D) over k, v (B, Tk, Hk, D): (out, lse),
    out (B, Tq, Hq, D) and lse float32 (B, Hq, Tq).

    ``scale`` None: 1 / sqrt(D).  ``softcap`` c (1e-30 to 1e30): scores
    c tanh(s / c).
    ``slopes`` float32 (Hq, axes) with ``pos_q`` (axes, B, Tq) and ``pos_k``
    (axes, B, Tk) int32: minus slope times distance, summed over 1 to 3
    axes.  ``kv_len`` int32 (B): keys in use, the queries the last Tq of
    them.  ``doc_offsets`` int32 (B, n + 1): documents packed in a row, each
    query seeing its own.  ``causal``, and with it ``prefix`` int32 (B, n) or
    (B): how many first tokens of a document (of the sequence) all its
    queries see.  A query that sees nothing gives 0 and -inf.
    ``out``: preallocated (out, lse); ``workspace``: a uint8 tensor of
    mp3d_attention_workspace_bytes(...) (None: allocated)."""
    lib = _lib.load()
    a = _attention(q, k, v, scale, softcap, causal, kv_len, doc_offsets, prefix, slopes, pos_q,
                   pos_k)
    B, Tq, Hq, _ = q.shape
    if out is None:
        o = torch.empty_like(q, memory_format=_contiguous)
        lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
        _same(o, "out", q.shape, q.dtype, q.device)
        _same(lse, "lse", (B, Hq, Tq), torch.float32, q.device)
    ws, n = _workspace(lib, a, 0, workspace, q.device)
    _lib.check(lib.mp3d_attention_forward(a, q.data_ptr(), k.data_ptr(),
                                          v.data_ptr(), o.data_ptr(), lse.data_ptr(), _ptr(ws), n,
                                          _stream(q)))
    return o, lse


def mp3d_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                            v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, *, scale=None,
                            softcap: float = 0.0, causal: bool = False,
                            kv_len: torch.Tensor | None = None,
                            doc_offsets: torch.Tensor | None = None,
                            prefix: torch.Tensor | None = None,
                            slopes: torch.Tensor | None = None,
                            pos_q: torch.Tensor | None = None,
                            pos_k: torch.Tensor | None = None, grads=None,
                            workspace: torch.Tensor | None = None):
    """(dq, dk, dv) from ``dout`` (B, Tq, Hq, D), the forward's inputs and
    keyword arguments, and its out and lse.  dk and dv are summed over the
    query heads that share a key head.  ``grads``: preallocated contiguous
    (dq, dk, dv).  The slopes are constants: they get no gradient."""
    lib = _lib.load()
    a = _attention(q, k, v, scale, softcap, causal, kv_len, doc_offsets, prefix, slopes, pos_q,
                   pos_k)
    shape, gs = _heads(dout, "dout", q)
    if shape != q.shape:
        raise ValueError("dout must have q's shape")
    _same(out, "out", q.shape, q.dtype, q.device)
    _same(lse, "lse", (q.shape[0], q.shape[2], q.shape[1]), torch.float32, q.device)
    if grads is None:
        dq = torch.empty_like(q, memory_format=_contiguous)
        dk = torch.empty_like(k, memory_format=_contiguous)
        dv = torch.empty_like(k, memory_format=_contiguous)
    else:
        dq, dk, dv = grads
        for t, like, n in ((dq, q, "dq"), (dk, k, "dk"), (dv, k, "dv")):
            _same(t, n, like.shape, q.dtype, q.device)
    ws, n = _workspace(lib, a, 1, workspace, q.device)
    _lib.check(lib.mp3d_attention_backward(a, dout.data_ptr(), _i64x3(*gs),
                                           q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                           out.data_ptr(), lse.data_ptr(), dq.data_ptr(),
                                           dk.data_ptr(), dv.data_ptr(), _ptr(ws), n, _stream(q)))
    return dq, dk, dv


# ------------------------------------------------------------------ gated norm

def _norm_args(x, h, gate, post_weight, pre_weight, norm, post_norm, pre_norm):
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous with the channels last")
    code = _code(x, "x")
    C = x.shape[-1]
    rows = x.numel() // C if C else 0
    if norm not in _NORM:
        raise ValueError("norm must be 'rms' or 'layer'")
    if h is not None:
        _same(h, "h", x.shape, x.dtype, x.device)
    for t, n in ((post_weight, "post_weight"), (pre_weight, "pre_weight")):
        if t is not None:
            _same(t, n, (C,), x.dtype, x.device)
    gate_rows = 0
    if gate is not None:
        if gate.dim() == 1:
            gate = gate[None]
        gate_rows = gate.shape[0]
        _same(gate, "gate", (gate_rows, C), x.dtype, x.device)
    parts = ((_lib.MP3D_NORM_POST if post_norm and h is not None else 0)
             | (_lib.MP3D_NORM_PRE if pre_norm else 0))
    return code, rows, C, gate_rows, parts


def mp3d_gated_norm_workspace_bytes(dtype: torch.dtype, rows: int, C: int,
                                    gate_rows: int = 0) -> int:
    """Workspace bytes of mp3d_gated_norm_backward."""
    nbytes = ctypes.c_size_t()
    _lib.check(_lib.load().mp3d_gated_norm_workspace_bytes(_DTYPE[dtype], rows, C, gate_rows,
                                                           ctypes.byref(nbytes)))
    return nbytes.value


def mp3d_gated_norm_forward(x: torch.Tensor, h: torch.Tensor | None = None, *,
                            gate: torch.Tensor | None = None,
                            post_weight: torch.Tensor | None = None,
                            pre_weight: torch.Tensor | None = None,
                            residual_scale: float = 1.0, norm: str = "rms", eps: float = 1e-6,
                            post_norm: bool = True, pre_norm: bool = True, out=None):
    """y = x + residual_scale * gate * post_weight * n(h), z = pre_weight * n(y):
    (y, z, stats).

    ``x`` (residual stream) and ``h`` (a block's output) are (..., C),
    contiguous.  ``h`` None: y is x itself (z = pre_weight * n(x)).  ``gate``
    (C) or (G, C), each row for 1/G of the rows; weights (C).  ``norm`` "rms"
    or "layer".  ``post_norm`` False: n(h) is h; ``pre_norm`` False: z is
    None.  ``stats`` is what the backward needs; ``out``: preallocated
    (y, z)."""
    lib = _lib.load()
    code, rows, C, gate_rows, parts = _norm_args(x, h, gate, post_weight, pre_weight, norm,
                                                 post_norm, pre_norm)
    y, z = (None, None) if out is None else out
    if h is None:
        y = None
    else:
        y = torch.empty_like(x) if y is None else _same(y, "y", x.shape, x.dtype, x.device)
    if not pre_norm:
        z = None
    else:
        z = torch.empty_like(x) if z is None else _same(z, "z", x.shape, x.dtype, x.device)
    stats = torch.empty((rows, 4), dtype=torch.float32, device=x.device)
    _lib.check(lib.mp3d_gated_norm_forward(
        x.data_ptr(), _ptr(h), _ptr(gate), _ptr(post_weight), _ptr(pre_weight), _ptr(y), _ptr(z),
        stats.data_ptr(), code, rows, C, gate_rows, float(residual_scale), _NORM[norm], parts,
        float(eps), _stream(x)))
    return (x if h is None else y), z, stats


def mp3d_gated_norm_backward(dy: torch.Tensor | None, dz: torch.Tensor | None, x: torch.Tensor,
                             h: torch.Tensor | None, stats: torch.Tensor, *,
                             gate: torch.Tensor | None = None,
                             post_weight: torch.Tensor | None = None,
                             pre_weight: torch.Tensor | None = None,
                             residual_scale: float = 1.0, norm: str = "rms", eps: float = 1e-6,
                             post_norm: bool = True, pre_norm: bool = True,
                             workspace: torch.Tensor | None = None):
    """(dx, dh, dgate, dpost_weight, dpre_weight) from the gradients of y
    (None: 0) and z; None in the place of what has no gradient.  dx and dh
    have x's dtype, the others are float32.  Arguments as for the forward."""
    lib = _lib.load()
    code, rows, C, gate_rows, parts = _norm_args(x, h, gate, post_weight, pre_weight, norm,
                                                 post_norm, pre_norm)
    for t, n in ((dy, "dy"), (dz, "dz")):
        if t is not None:
            _same(t, n, x.shape, x.dtype, x.device)
    if pre_norm and dz is None:
        raise ValueError("dz is needed (pre_norm)")
    _same(stats, "stats", (rows, 4), torch.float32, x.device)
    new = lambda *shape: torch.empty(shape, dtype=torch.float32, device=x.device)  # noqa: E731
    dx = torch.empty_like(x)
    dh = None if h is None else torch.empty_like(x)
    dgate = None if gate is None else new(gate_rows, C).view(gate.shape)
    dpost = None if post_weight is None else new(C)
    dpre = None if pre_weight is None else new(C)
    nbytes = ctypes.c_size_t()
    _lib.check(lib.mp3d_gated_norm_workspace_bytes(code, rows, C, gate_rows,
                                                   ctypes.byref(nbytes)))
    ws, n = _lend(nbytes.value, workspace, x.device)
    _lib.check(lib.mp3d_gated_norm_backward(
        _ptr(dy), _ptr(dz) if pre_norm else None, x.data_ptr(), _ptr(h), _ptr(gate),
        _ptr(post_weight), _ptr(pre_weight), stats.data_ptr(), dx.data_ptr(), _ptr(dh),
        _ptr(dgate), _ptr(dpost), _ptr(dpre), code, rows, C, gate_rows, float(residual_scale),
        _NORM[norm], parts, float(eps), _ptr(ws), n, _stream(x)))
    return dx, dh, dgate, dpost, dpre
