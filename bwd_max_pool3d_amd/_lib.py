"""ctypes view of libmp3d.so (declared in include/mp3d.h).

Loading fails loudly: there is no fallback implementation anywhere in this
package, so a missing or unloadable library is an ImportError for every op.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libmp3d.so")

(MP3D_OK, MP3D_EINVAL, MP3D_EDTYPE, MP3D_ENOTDIV, MP3D_EOVERFLOW, MP3D_EHIP,
 MP3D_EWORKSPACE) = range(7)
MP3D_F32, MP3D_F16, MP3D_BF16, MP3D_F64 = 0, 1, 2, 3

MP3D_IDX_NONE, MP3D_IDX_I32, MP3D_IDX_I64 = -1, 0, 1

EXPORTS = ("mp3d_forward", "amp3d_forward", "mp3d_backward", "mp3d_out_size",
           "mp3d_out_size_ex", "mp3d_forward_ex", "mp3d_backward_ex", "mp3d_backward_recompute",
           "mp3d_recompute_workspace_size", "mp3d_backward_recompute_ws",
           "mp3d_backward_workspace_bytes", "mp3d_time_next_call",
           "mp3d_backward_recompute_static", "mp3d_strerror", "mp3d_last_error",
           "mp3d_rope_forward", "mp3d_rope_backward", "mp3d_attention_workspace_bytes",
           "mp3d_attention_forward", "mp3d_attention_backward", "mp3d_gated_norm_forward",
           "mp3d_gated_norm_workspace_bytes", "mp3d_gated_norm_backward")

MP3D_NORM_RMS, MP3D_NORM_LAYER = 0, 1
MP3D_NORM_POST, MP3D_NORM_PRE = 1, 2

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_lib = None


class Attention(ctypes.Structure):
    """struct mp3d_attention (include/mp3d.h)."""
    _fields_ = [("dtype", ctypes.c_int), ("B", _i64), ("Tq", _i64), ("Tk", _i64), ("Hq", _i32),
                ("Hk", _i32), ("D", _i32), ("q_stride", _i64 * 3), ("k_stride", _i64 * 3),
                ("v_stride", _i64 * 3), ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("causal", ctypes.c_int), ("kv_len", _vp), ("doc_offsets", _vp),
                ("n_docs", _i32), ("prefix", _vp), ("axes", _i32), ("slopes", _vp),
                ("pos_q", _vp), ("pos_k", _vp)]


class Mp3dError(RuntimeError):
    """A libmp3d call returned a non-zero status."""

    def __init__(self, code: int, message: str):
        super().__init__("%s (status %d)" % (message, code))
        self.code = code


def load(path: str | None = None) -> ctypes.CDLL:
    """The loaded library (cached).  Raises ImportError if it is missing.
    ``MP3D_LIBRARY`` in the environment names another build of the same
    library (for comparing builds); the default is the in-tree one."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = os.environ.get("MP3D_LIBRARY") or LIBRARY
    if not os.path.exists(path):
        raise ImportError(
            "libmp3d.so is not built at %s; run `python -m bwd_max_pool3d_amd._build` "
            "(or __graft_entry__.build()) first" % path)
    lib = ctypes.CDLL(path)
    lib.mp3d_forward.argtypes = [_vp, _vp, _vp, ctypes.c_int] + [_i64] * 5 + [_i32] * 6 + [_vp]
    lib.amp3d_forward.argtypes = [_vp, _vp, _vp, ctypes.c_int] + [_i64] * 5 + [_i32] * 3 + [_vp]
    lib.mp3d_backward.argtypes = ([_vp, _vp, _vp, ctypes.c_int] + [_i64] * 5 + [_i32] * 9
                                  + [ctypes.c_int, _vp])
    lib.mp3d_out_size.argtypes = [_i64, _i32, _i32, ctypes.POINTER(_i64)]
    _a3 = ctypes.POINTER(_i32)
    lib.mp3d_out_size_ex.argtypes = [_i64, _i32, _i32, _i32, _i32, ctypes.c_int,
                                     ctypes.POINTER(_i64)]
    lib.mp3d_forward_ex.argtypes = ([_vp, _vp, _vp, ctypes.c_int, ctypes.c_int] + [_i64] * 5
                                    + [_i32] * 3 + [_a3] * 4 + [_vp])
    lib.mp3d_backward_ex.argtypes = ([_vp, _vp, _vp, ctypes.c_int, ctypes.c_int] + [_i64] * 5
                                     + [_i32] * 3 + [_a3] * 4 + [ctypes.c_int, _vp])
    lib.mp3d_backward_recompute.argtypes = ([_vp, _vp, _vp, _vp, ctypes.c_int] + [_i64] * 5
                                            + [_i32] * 3 + [_a3] * 4 + [ctypes.c_int, _vp])
    lib.mp3d_recompute_workspace_size.argtypes = ([ctypes.c_int] + [_i64] * 2 + [_i32] * 3
                                                  + [ctypes.POINTER(ctypes.c_size_t)])
    lib.mp3d_backward_recompute_ws.argtypes = ([_vp, _vp, _vp, _vp, ctypes.c_int] + [_i64] * 5
                                               + [_i32] * 3 + [_a3] * 4
                                               + [ctypes.c_int, _vp, ctypes.c_size_t, _vp])
    lib.mp3d_backward_workspace_bytes.argtypes = ([ctypes.c_int] * 2 + [_i64] * 2 + [_i32] * 3
                                                  + [ctypes.POINTER(ctypes.c_size_t)])
    lib.mp3d_time_next_call.argtypes = [_vp, _vp]
    lib.mp3d_backward_recompute_static.argtypes = ([_vp, _vp, _vp, _vp, ctypes.c_int]
                                                   + [_i64] * 5 + [_i32] * 3 + [_a3] * 4
                                                   + [ctypes.c_int, _vp])
    # (host arrays and the attention descriptor as void*: ctypes objects and
    # packed bytes are both taken)
    _f32, _int, _size = ctypes.c_float, ctypes.c_int, ctypes.c_size_t
    for name in ("mp3d_rope_forward", "mp3d_rope_backward"):
        getattr(lib, name).argtypes = ([_vp] * 4 + [_int] + [_i64] * 2 + [_i32] * 3 + [_vp] * 4
                                       + [_vp] * 4 + [_int, _vp])
    _attn = _vp
    lib.mp3d_attention_workspace_bytes.argtypes = [_attn, _int, ctypes.POINTER(_size)]
    lib.mp3d_attention_forward.argtypes = [_attn] + [_vp] * 6 + [_size, _vp]
    lib.mp3d_attention_backward.argtypes = [_attn] + [_vp] * 11 + [_size, _vp]
    lib.mp3d_gated_norm_forward.argtypes = ([_vp] * 8 + [_int, _i64, _i32, _i64, _f32, _int, _int,
                                                        _f32, _vp])
    lib.mp3d_gated_norm_workspace_bytes.argtypes = [_int, _i64, _i32, _i64,
                                                    ctypes.POINTER(_size)]
    lib.mp3d_gated_norm_backward.argtypes = ([_vp] * 13 + [_int, _i64, _i32, _i64, _f32, _int,
                                                          _int, _f32, _vp, _size, _vp])
    lib.mp3d_strerror.argtypes = [ctypes.c_int]
    lib.mp3d_strerror.restype = ctypes.c_char_p
    lib.mp3d_last_error.argtypes = []
    lib.mp3d_last_error.restype = ctypes.c_char_p
    for name in ("mp3d_forward", "amp3d_forward", "mp3d_backward", "mp3d_out_size",
                 "mp3d_out_size_ex", "mp3d_forward_ex", "mp3d_backward_ex",
                 "mp3d_backward_recompute", "mp3d_recompute_workspace_size",
                 "mp3d_backward_recompute_ws", "mp3d_backward_workspace_bytes",
                 "mp3d_time_next_call", "mp3d_backward_recompute_static", "mp3d_rope_forward",
                 "mp3d_rope_backward", "mp3d_attention_workspace_bytes",
                 "mp3d_attention_forward", "mp3d_attention_backward", "mp3d_gated_norm_forward",
                 "mp3d_gated_norm_workspace_bytes", "mp3d_gated_norm_backward"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def check(code: int) -> None:
    if code != MP3D_OK:
        lib = load()
        msg = lib.mp3d_last_error().decode() or lib.mp3d_strerror(code).decode()
        raise Mp3dError(code, msg)
