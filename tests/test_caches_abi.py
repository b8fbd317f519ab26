"""The C ABI of caches and of attention over them, on the host: bad arguments
are refused with the documented codes before anything touches the GPU."""
import ctypes

import pytest
import torch

import bwd_max_pool3d_amd as mp
from bwd_max_pool3d_amd import _lib, caches

FAKE = 0x1000   # never dereferenced: every call below fails validation or has nothing to do
A3 = ctypes.c_int64 * 3
E, W, D_, V = _lib.MP3D_EINVAL, _lib.MP3D_EWORKSPACE, _lib.MP3D_EDTYPE, _lib.MP3D_EOVERFLOW


def cache(B=2, T=16, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, st=(512, 32, 16), sst=(32, 2, 1)):
    c = _lib.Cache()
    c.B, c.T, c.k, c.v, c.k_scale, c.v_scale = B, T, k, v, ks, vs
    c.k_stride, c.v_stride = A3(*st), A3(*st)
    c.k_scale_stride, c.v_scale_stride = A3(*sst), A3(*sst)
    return c


def write(c=None, *, format=1, k=FAKE, v=FAKE, dtype=0, T=4, H=2, D=16, st=(128, 32, 16), null=False):
    st = None if st is None else A3(*st)
    return _lib.load().mp3d_cache_write(None if null else ctypes.byref(c or cache()), format, k, v,
                                        dtype, T, H, D, st, st, None, None, None)


def read(c=None, *, format=1, k=FAKE, v=FAKE, dtype=0, T=4, H=2, D=16):
    return _lib.load().mp3d_cache_read(ctypes.byref(c or cache()), format, k, v, dtype, T, H, D,
                                       None, None, None)


BOTH = [(dict(format=0), E), (dict(format=3), E), (dict(format=-1), E), (dict(dtype=3), D_),
        (dict(T=-1), E), (dict(H=0), E), (dict(H=70000), E), (dict(D=0), E), (dict(D=1025), E),
        (dict(T=1 << 31), V), (dict(k=None), E), (dict(v=None), E), (dict(k=FAKE + 1), E),
        (dict(c=cache(B=-1)), E), (dict(c=cache(T=-1)), E), (dict(c=cache(T=1 << 31)), V),
        (dict(c=cache(B=1 << 30, T=1 << 20)), V), (dict(c=cache(k=None)), E),
        (dict(c=cache(vs=None)), E), (dict(c=cache(st=(512, -32, 16))), E),
        (dict(c=cache(sst=(32, 2, -1))), E)]


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("how,code", BOTH, ids=lambda v: str(v)[:50])
def test_cache_refusals(call, how, code):
    assert call(**how) == code
    assert _lib.load().mp3d_last_error().decode() != ""


def test_write_refusals():
    assert write(null=True) == E
    assert write(st=None) == E
    assert write(st=(128, -1, 16)) == E
    # sequences, rows or heads that share their bytes cannot be written
    for st in ((0, 32, 16), (512, 0, 16), (512, 32, 0)):
        assert write(cache(st=st)) == E
    for st in ((0, 2, 1), (32, 0, 1), (32, 2, 0)):
        assert write(cache(sst=st)) == E
    assert read(k=FAKE + 8) == E                           # outputs are 16-byte aligned


def test_cache_nothing_to_do():
    assert write(T=0, k=None) == _lib.MP3D_OK
    assert write(cache(B=0), k=None) == _lib.MP3D_OK
    assert write(cache(T=0, k=None), k=None) == _lib.MP3D_OK
    assert read(T=0, k=None) == _lib.MP3D_OK
    assert read(cache(B=0), k=None) == _lib.MP3D_OK


def desc(**over):
    a = _lib.AttentionCache()
    a.dtype, a.format, a.B, a.Tq, a.Hq, a.Hk, a.D, a.causal = 0, 1, 2, 4, 4, 2, 16, 1
    a.q_stride = A3(256, 64, 16)
    a.scale = 1.0
    a.own, a.prefix = cache(), cache(B=1)
    for n, v in over.items():
        setattr(a, n, v)
    return a


DESC = [
    (dict(dtype=3), D_), (dict(format=3), E), (dict(format=-1), E), (dict(B=-1), E), (dict(Tq=-1), E),
    (dict(Hk=0), E), (dict(Hq=3), E), (dict(D=0), E), (dict(D=129), E), (dict(causal=2), E),
    (dict(own=cache(B=3)), E), (dict(own=cache(T=-1)), E), (dict(own=cache(T=1 << 31)), V),
    (dict(prefix=cache(B=-1)), E), (dict(B=3, own=cache(B=3), prefix=cache(B=2)), E),
    (dict(prefix=cache(B=4)), E), (dict(Tq=1 << 31), V), (dict(Tq=1 << 29), V),
    (dict(softcap=-1.0), E), (dict(softcap=float("nan")), E), (dict(softcap=1e31), E),
    (dict(scale=float("nan")), E), (dict(scale=float("inf")), E), (dict(axes=4), E),
    (dict(axes=1), E), (dict(axes=1, slopes=FAKE, pos_q=FAKE), E),
    (dict(axes=1, slopes=FAKE, pos_q=FAKE, pos_k=FAKE), E),       # a prefix has positions too
    (dict(q_stride=A3(256, -64, 16)), E), (dict(own=cache(st=(512, -32, 16))), E),
]


@pytest.mark.parametrize("over,code", DESC, ids=lambda v: str(v)[:50])
def test_attention_descriptor_refusals(over, code):
    lib, n = _lib.load(), ctypes.c_size_t()
    a = ctypes.byref(desc(**over))
    assert lib.mp3d_attention_cached_workspace_bytes(a, ctypes.byref(n)) == code
    assert lib.mp3d_attention_cached(a, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == code
    assert lib.mp3d_last_error().decode() != ""


def test_attention_call_refusals():
    lib, n = _lib.load(), ctypes.c_size_t()
    call = lambda a, *t, ws=FAKE, nb=1 << 40: lib.mp3d_attention_cached(  # noqa: E731
        ctypes.byref(a), *t, ws, nb, None)
    a = desc()
    assert lib.mp3d_attention_cached_workspace_bytes(ctypes.byref(a), None) == E
    assert lib.mp3d_attention_cached_workspace_bytes(None, ctypes.byref(n)) == E
    assert call(a, None, FAKE, FAKE) == E
    assert call(a, FAKE, None, FAKE) == E
    assert call(a, FAKE, FAKE, None) == E
    assert call(a, FAKE, FAKE + 8, FAKE) == E              # out is 16-byte aligned
    assert call(a, FAKE + 1, FAKE, FAKE) == E
    for part in (dict(own=cache(k=None)), dict(own=cache(vs=None)), dict(prefix=cache(B=1, v=None))):
        assert call(desc(**part), FAKE, FAKE, FAKE) == E
    plain = dict(format=0, own=cache(k=FAKE + 2), prefix=cache(B=0))
    assert call(desc(**plain), FAKE, FAKE, FAKE) == E
    assert lib.mp3d_attention_cached_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value > 0                                     # prefix and own cache are joined
    assert call(a, FAKE, FAKE, FAKE, ws=None) == W
    assert call(a, FAKE, FAKE, FAKE, nb=n.value - 1) == W
    assert call(a, FAKE, FAKE, FAKE, ws=FAKE + 4) == W


def test_attention_nothing_to_do():
    lib = _lib.load()
    for a in (desc(B=0, own=cache(B=0), prefix=cache(B=0)), desc(Tq=0)):
        assert lib.mp3d_attention_cached(ctypes.byref(a), None, None, None, None, 0,
                                         None) == _lib.MP3D_OK


def test_packed_structures_have_the_declared_size():
    assert len(caches._cache_struct(*[0] * 18)) == ctypes.sizeof(_lib.Cache)
    n = len(caches._attention_struct(*[0] * 11, 0.0, 0.0, *[0] * 36, *[0] * 7))
    assert n == ctypes.sizeof(_lib.AttentionCache)


def test_python_names_and_refusals():
    for name in caches.__all__:
        assert name in mp.__all__ and callable(getattr(mp, name))
    x = torch.zeros(1, 2, 2, 8)
    c = mp.mp3d_cache_empty(1, 4, 2, 8, "e4m3", device="cpu")
    assert [tuple(t.shape) for t in c] == [(1, 4, 2, 8), (1, 4, 2, 1)] * 2
    c4 = mp.mp3d_cache_empty(1, 4, 2, 33, "e2m1", device="cpu")
    assert [tuple(t.shape) for t in c4] == [(1, 4, 2, 17), (1, 4, 2, 2)] * 2
    with pytest.raises(ValueError):
        mp.mp3d_cache_empty(1, 4, 2, 8, None, device="cpu")
    with pytest.raises(ValueError):
        mp.mp3d_cache_write(x, x, c, "e4m3")               # host tensors
    with pytest.raises(ValueError):
        mp.mp3d_cache_read(c, "e4m3", 8, torch.float32)
    with pytest.raises(ValueError):
        mp.mp3d_attention_cached(x, c, format="e4m3")
    with pytest.raises(ValueError):
        mp.mp3d_cache_read(c, "int8", 8, torch.float32)
