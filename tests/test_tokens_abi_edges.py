"""The token operators' C ABI on the host, at the ends of its ranges."""
import ctypes

import pytest

from bwd_max_pool3d_amd import _lib
from test_tokens_abi import A3, FAKE, ST, desc


@pytest.mark.parametrize("over", [dict(), dict(Tk=300, doc_offsets=FAKE, n_docs=2),
                                  dict(axes=2, slopes=FAKE, pos_q=FAKE, pos_k=FAKE),
                                  dict(Hq=2), dict(Tk=0), dict(B=0), dict(Tq=7)], ids=str)
def test_backward_takes_the_workspace_it_asks_for(over):
    """A workspace of the queried size is not refused for its size; one byte
    less is, wherever some is needed."""
    lib, n = _lib.load(), ctypes.c_size_t()
    how = dict(Tq=0)
    how.update(over)
    a = ctypes.byref(desc(**how))
    assert lib.mp3d_attention_workspace_bytes(a, 1, ctypes.byref(n)) == _lib.MP3D_OK

    def call(nbytes, stride):
        return lib.mp3d_attention_backward(a, FAKE, stride, *[FAKE] * 8, FAKE, nbytes, None)

    if n.value:
        assert call(n.value - 1, A3(*ST)) == _lib.MP3D_EWORKSPACE
        assert "%d bytes" % n.value in _lib.load().mp3d_last_error().decode()
    if how["Tq"] == 0 and how.get("Tk", 4) and how.get("B", 2):
        # shared heads, documents and a bias take some even without queries
        assert n.value > 0 or how.get("Hq", 4) == 2 or "doc_offsets" in how
    else:
        assert (n.value > 0) == (how["Tq"] > 0)


@pytest.mark.parametrize("over,code", [
    (dict(Tq=0, pos_k=FAKE), _lib.MP3D_OK), (dict(Tk=0, pos_q=FAKE), _lib.MP3D_OK),
    (dict(Tq=0, Tk=0), _lib.MP3D_OK), (dict(B=0), _lib.MP3D_OK),
    (dict(pos_k=FAKE), _lib.MP3D_EINVAL), (dict(pos_q=FAKE), _lib.MP3D_EINVAL),
    (dict(Tq=0), _lib.MP3D_EINVAL), (dict(Tk=0), _lib.MP3D_EINVAL)], ids=str)
def test_positions_of_no_tokens_may_be_null(over, code):
    lib, n = _lib.load(), ctypes.c_size_t()
    a = ctypes.byref(desc(axes=1, slopes=FAKE, **over))
    for backward in (0, 1):
        assert lib.mp3d_attention_workspace_bytes(a, backward, ctypes.byref(n)) == code


@pytest.mark.parametrize("cap,code", [(0.0, _lib.MP3D_OK), (1e-30, _lib.MP3D_OK),
                                      (1e30, _lib.MP3D_OK), (1e-31, _lib.MP3D_EINVAL),
                                      (1e-42, _lib.MP3D_EINVAL), (1e31, _lib.MP3D_EINVAL)])
def test_range_of_caps(cap, code):
    n = ctypes.c_size_t()
    a = ctypes.byref(desc(softcap=cap))
    assert _lib.load().mp3d_attention_workspace_bytes(a, 1, ctypes.byref(n)) == code
