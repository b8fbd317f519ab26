"""The token operators' C ABI on the host: bad arguments are refused with the
documented codes before anything touches the GPU."""
import ctypes

import pytest

import bwd_max_pool3d_amd as mp
from bwd_max_pool3d_amd import _lib

FAKE = 0x1000   # never dereferenced: every call below fails validation or has nothing to do
A3 = ctypes.c_int64 * 3
I3 = ctypes.c_int32 * 3
ST = (64, 32, 8)


def rope(*, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, dtype=0, B=2, T=6, Hq=2, Hk=1, D=8, qs=ST, freq=FAKE,
         pairs=(1, 1, 2), pos=None, grid=(1, 2, 3), il=0, name="mp3d_rope_forward"):
    st = None if qs is None else A3(*qs)
    return getattr(_lib.load(), name)(
        q, k, qo, ko, dtype, B, T, Hq, Hk, D, st, A3(*ST), A3(*ST), A3(*ST), freq,
        None if pairs is None else I3(*pairs), pos, None if grid is None else I3(*grid), il, None)


@pytest.mark.parametrize("name", ["mp3d_rope_forward", "mp3d_rope_backward"])
@pytest.mark.parametrize("how,code", [
    (dict(dtype=3), _lib.MP3D_EDTYPE), (dict(dtype=-1), _lib.MP3D_EDTYPE),
    (dict(B=-1), _lib.MP3D_EINVAL), (dict(T=-1), _lib.MP3D_EINVAL),
    (dict(Hq=-1), _lib.MP3D_EINVAL), (dict(Hk=70000), _lib.MP3D_EINVAL),
    (dict(D=0), _lib.MP3D_EINVAL), (dict(D=70000), _lib.MP3D_EINVAL),
    (dict(T=1 << 31, grid=None, pos=FAKE), _lib.MP3D_EOVERFLOW),
    (dict(B=1 << 20, T=1 << 20, grid=None, pos=FAKE), _lib.MP3D_EOVERFLOW),
    (dict(pairs=None), _lib.MP3D_EINVAL), (dict(pairs=(-1, 1, 1)), _lib.MP3D_EINVAL),
    (dict(pairs=(2, 2, 1)), _lib.MP3D_EINVAL), (dict(il=2), _lib.MP3D_EINVAL),
    (dict(pos=FAKE), _lib.MP3D_EINVAL), (dict(grid=None), _lib.MP3D_EINVAL),
    (dict(grid=(1, 2, 4)), _lib.MP3D_EINVAL), (dict(grid=(0, 2, 3)), _lib.MP3D_EINVAL),
    (dict(grid=(1 << 20, 1 << 20, 1)), _lib.MP3D_EINVAL),
    (dict(freq=None), _lib.MP3D_EINVAL), (dict(q=None), _lib.MP3D_EINVAL),
    (dict(ko=None), _lib.MP3D_EINVAL), (dict(qs=None), _lib.MP3D_EINVAL),
    (dict(qs=(64, -32, 8)), _lib.MP3D_EINVAL), (dict(q=FAKE + 1), _lib.MP3D_EINVAL),
], ids=str)
def test_rope_refusals(name, how, code):
    assert rope(name=name, **how) == code
    assert _lib.load().mp3d_last_error().decode() != ""


def test_rope_nothing_to_do():
    assert rope(B=0, q=None, k=None, qo=None, ko=None) == _lib.MP3D_OK
    assert rope(T=0, grid=None, q=None, freq=None) == _lib.MP3D_OK
    assert rope(Hq=0, Hk=0) == _lib.MP3D_OK


def norm(*, x=FAKE, h=FAKE, gate=None, post=None, pre=None, y=FAKE, z=FAKE, stats=FAKE, dtype=0,
         rows=4, C=8, gr=0, kind=0, parts=3, eps=1e-6):
    return _lib.load().mp3d_gated_norm_forward(x, h, gate, post, pre, y, z, stats, dtype, rows, C,
                                               gr, 1.0, kind, parts, eps, None)


def norm_back(*, dy=FAKE, dz=FAKE, x=FAKE, h=FAKE, gate=None, post=None, pre=None, stats=FAKE,
              dx=FAKE, dh=FAKE, dgate=None, dpost=None, dpre=None, dtype=0, rows=4, C=8, gr=0,
              kind=0, parts=3, ws=FAKE, n=1 << 30):
    return _lib.load().mp3d_gated_norm_backward(dy, dz, x, h, gate, post, pre, stats, dx, dh, dgate,
                                                dpost, dpre, dtype, rows, C, gr, 1.0, kind, parts,
                                                1e-6, ws, n, None)


@pytest.mark.parametrize("call,code", [
    (lambda: norm(dtype=3), _lib.MP3D_EDTYPE), (lambda: norm(rows=-1), _lib.MP3D_EINVAL),
    (lambda: norm(C=0), _lib.MP3D_EINVAL), (lambda: norm(C=16385), _lib.MP3D_EINVAL),
    (lambda: norm(rows=1 << 31), _lib.MP3D_EOVERFLOW), (lambda: norm(kind=2), _lib.MP3D_EINVAL),
    (lambda: norm(parts=4), _lib.MP3D_EINVAL), (lambda: norm(eps=-1.0), _lib.MP3D_EINVAL),
    (lambda: norm(eps=float("nan")), _lib.MP3D_EINVAL), (lambda: norm(x=None), _lib.MP3D_EINVAL),
    (lambda: norm(h=None), _lib.MP3D_EINVAL),                      # a post norm without h
    (lambda: norm(h=None, parts=0), _lib.MP3D_EINVAL),
    (lambda: norm(h=None, parts=2, gate=FAKE, gr=1), _lib.MP3D_EINVAL),
    (lambda: norm(parts=1, pre=FAKE), _lib.MP3D_EINVAL),
    (lambda: norm(gate=FAKE, gr=0), _lib.MP3D_EINVAL),
    (lambda: norm(gate=FAKE, gr=3), _lib.MP3D_EINVAL),
    (lambda: norm(y=None), _lib.MP3D_EINVAL), (lambda: norm(z=None), _lib.MP3D_EINVAL),
    (lambda: norm(x=FAKE + 2), _lib.MP3D_EINVAL), (lambda: norm(stats=FAKE + 4), _lib.MP3D_EINVAL),
    (lambda: norm_back(stats=None), _lib.MP3D_EINVAL),
    (lambda: norm_back(dz=None), _lib.MP3D_EINVAL), (lambda: norm_back(dx=None), _lib.MP3D_EINVAL),
    (lambda: norm_back(dh=None), _lib.MP3D_EINVAL),
    (lambda: norm_back(gate=FAKE, gr=2), _lib.MP3D_EINVAL),        # dgate goes with gate
    (lambda: norm_back(dgate=FAKE), _lib.MP3D_EINVAL),
    (lambda: norm_back(dpost=FAKE), _lib.MP3D_EINVAL),
    (lambda: norm_back(dpre=FAKE), _lib.MP3D_EINVAL),
    (lambda: norm_back(ws=None), _lib.MP3D_EWORKSPACE),
    (lambda: norm_back(n=16), _lib.MP3D_EWORKSPACE),
    (lambda: norm_back(ws=FAKE + 8), _lib.MP3D_EWORKSPACE),
])
def test_norm_refusals(call, code):
    assert call() == code
    assert _lib.load().mp3d_last_error().decode() != ""


def test_norm_nothing_to_do():
    assert norm(rows=0, x=None, h=None, y=None, z=None, stats=None) == _lib.MP3D_OK
    assert norm_back(rows=0, x=None, h=None, dz=None, stats=None, dx=None) == _lib.MP3D_OK


def desc(**over):
    a = _lib.Attention()
    a.dtype, a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.D = 0, 2, 4, 4, 4, 2, 8
    for n in ("q_stride", "k_stride", "v_stride"):
        setattr(a, n, A3(128, 32, 8))
    a.scale = 1.0
    for n, v in over.items():
        setattr(a, n, v)
    return a


DESC = [
    (dict(dtype=3), _lib.MP3D_EDTYPE), (dict(B=-1), _lib.MP3D_EINVAL),
    (dict(Tk=-1), _lib.MP3D_EINVAL), (dict(Hk=0), _lib.MP3D_EINVAL),
    (dict(Hq=3), _lib.MP3D_EINVAL), (dict(D=0), _lib.MP3D_EINVAL),
    (dict(D=129), _lib.MP3D_EINVAL), (dict(Tq=1 << 31), _lib.MP3D_EOVERFLOW),
    (dict(Tk=1 << 31), _lib.MP3D_EOVERFLOW), (dict(Tq=1 << 30), _lib.MP3D_EOVERFLOW),
    (dict(B=1 << 30, Tk=1 << 20), _lib.MP3D_EOVERFLOW), (dict(causal=2), _lib.MP3D_EINVAL),
    (dict(softcap=-1.0), _lib.MP3D_EINVAL), (dict(softcap=float("inf")), _lib.MP3D_EINVAL),
    (dict(softcap=float("nan")), _lib.MP3D_EINVAL), (dict(scale=float("nan")), _lib.MP3D_EINVAL),
    (dict(scale=float("-inf")), _lib.MP3D_EINVAL), (dict(prefix=FAKE), _lib.MP3D_EINVAL),
    (dict(doc_offsets=FAKE), _lib.MP3D_EINVAL), (dict(axes=4), _lib.MP3D_EINVAL),
    (dict(axes=1), _lib.MP3D_EINVAL), (dict(axes=1, slopes=FAKE, pos_q=FAKE), _lib.MP3D_EINVAL),
    (dict(k_stride=A3(128, -32, 8)), _lib.MP3D_EINVAL),
]


@pytest.mark.parametrize("over,code", DESC, ids=lambda v: str(v)[:60])
def test_attention_descriptor_refusals(over, code):
    lib, n = _lib.load(), ctypes.c_size_t()
    a = ctypes.byref(desc(**over))
    assert lib.mp3d_attention_workspace_bytes(a, 0, ctypes.byref(n)) == code
    assert lib.mp3d_attention_forward(a, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None) == code
    assert lib.mp3d_attention_backward(a, FAKE, A3(*ST), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                       FAKE, FAKE, 1 << 40, None) == code
    assert lib.mp3d_last_error().decode() != ""


def test_attention_call_refusals():
    lib, n = _lib.load(), ctypes.c_size_t()
    a = ctypes.byref(desc())
    E, W = _lib.MP3D_EINVAL, _lib.MP3D_EWORKSPACE
    assert lib.mp3d_attention_workspace_bytes(a, 0, None) == E
    assert lib.mp3d_attention_workspace_bytes(None, 0, ctypes.byref(n)) == E
    fwd = lambda *t, ws=None, nb=0, d=a: lib.mp3d_attention_forward(d, *t, ws, nb, None)  # noqa: E731
    assert fwd(None, FAKE, FAKE, FAKE, FAKE) == E
    assert fwd(FAKE, None, FAKE, FAKE, FAKE) == E
    assert fwd(FAKE, FAKE, FAKE, None, FAKE) == E
    assert fwd(FAKE, FAKE, FAKE, FAKE, None) == E
    assert fwd(FAKE, FAKE, FAKE, FAKE + 8, FAKE) == E              # out is 16-byte aligned
    assert fwd(FAKE + 1, FAKE, FAKE, FAKE, FAKE) == E
    long = ctypes.byref(desc(Tq=1, Tk=100000))
    assert lib.mp3d_attention_workspace_bytes(long, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert fwd(FAKE, FAKE, FAKE, FAKE, FAKE, d=long) == W
    assert fwd(FAKE, FAKE, FAKE, FAKE, FAKE, ws=FAKE, nb=n.value - 1, d=long) == W
    assert fwd(FAKE, FAKE, FAKE, FAKE, FAKE, ws=FAKE + 4, nb=n.value, d=long) == W
    bwd = lambda *t, ws=FAKE, nb=1 << 40, st=A3(*ST): lib.mp3d_attention_backward(  # noqa: E731
        a, t[0], st, *t[1:], ws, nb, None)
    ten = [FAKE] * 9
    for i in range(9):
        assert bwd(*ten[:i], None, *ten[i + 1:]) == E, i
    assert bwd(*ten, st=None) == E
    assert bwd(*ten, ws=None) == W
    assert bwd(*ten, nb=8) == W


def test_attention_nothing_to_do():
    lib = _lib.load()
    for d in (desc(B=0), desc(Tq=0)):
        assert lib.mp3d_attention_forward(ctypes.byref(d), None, None, None, None, None, None, 0,
                                          None) == _lib.MP3D_OK
    for d in (desc(B=0), desc(Tq=0, Tk=0)):
        assert lib.mp3d_attention_backward(ctypes.byref(d), *[None] * 11, 0, None) == _lib.MP3D_OK


def test_python_names():
    for name in ("mp3d_rope_forward", "mp3d_rope_backward", "mp3d_attention_forward",
                 "mp3d_attention_backward", "mp3d_attention_workspace_bytes",
                 "mp3d_gated_norm_forward", "mp3d_gated_norm_backward",
                 "mp3d_gated_norm_workspace_bytes"):
        assert name in mp.__all__ and callable(getattr(mp, name))


def test_python_refuses_host_tensors():
    import torch
    x = torch.zeros(1, 2, 2, 8)
    f = torch.ones(4)
    with pytest.raises(ValueError):
        mp.mp3d_rope_forward(x, x, f, (4, 0, 0), grid=(1, 1, 2))
    with pytest.raises(ValueError):
        mp.mp3d_attention_forward(x, x, x)
    with pytest.raises(ValueError):
        mp.mp3d_gated_norm_forward(x, x)


def test_norm_workspace_is_bounded():
    """The sums' workspace does not grow with the rows or the gate's rows."""
    import torch
    few = mp.mp3d_gated_norm_workspace_bytes(torch.bfloat16, 1 << 14, 1024, 1)
    many = mp.mp3d_gated_norm_workspace_bytes(torch.bfloat16, 1 << 24, 1024, 1 << 24)
    assert 0 < few <= many <= 1024 * 3 * 1024 * 4
    assert mp.mp3d_gated_norm_workspace_bytes(torch.float32, 0, 8) == 0
