"""The C ABI of attention over caches, on the host, at its ends: a prefix that
is not there, and what a workspace's size depends on."""
import ctypes

import pytest

from bwd_max_pool3d_amd import _lib

FAKE = 0x1000   # never dereferenced: these calls only size a workspace
A3 = ctypes.c_int64 * 3


def cache(B, T, H, D, at=FAKE):
    """Plain or e4m3 rows, head by head, starting at `at`."""
    c = _lib.Cache()
    c.B, c.T, c.k, c.v, c.k_scale, c.v_scale = B, T, at, at, FAKE, FAKE
    c.k_stride = c.v_stride = A3(H * T * D, D, T * D)
    c.k_scale_stride = c.v_scale_stride = A3(H * T * 4, 4, T * 4)
    return c


def desc(B, Tq, T, Hq, Hk, D, *, N=0, P=0, format=1, at=FAKE, kv_len=None):
    a = _lib.AttentionCache()
    a.dtype, a.format, a.B, a.Tq, a.Hq, a.Hk, a.D, a.causal = 2, format, B, Tq, Hq, Hk, D, 1
    a.q_stride = A3(Tq * Hq * D, Hq * D, D)
    a.scale = 1.0
    a.own, a.prefix, a.kv_len = cache(B, T, Hk, D, at), cache(N, P, Hk, D, at), kv_len
    return a


def size(a):
    n = ctypes.c_size_t()
    assert _lib.load().mp3d_attention_cached_workspace_bytes(
        ctypes.byref(a), ctypes.byref(n)) == _lib.MP3D_OK
    return n.value


@pytest.mark.parametrize("T", [0, 100, 8000])
def test_no_prefix_has_no_rows(T):
    """prefix.B = 0 is no prefix, whatever its T says: 40 rows a key head over
    caches of 8000 were cut as if a prefix of 16500 rows were there."""
    without = size(desc(2, 10, T, 8, 2, 32))
    for P in (1, 70, 16500):
        assert size(desc(2, 10, T, 8, 2, 32, P=P)) == without


@pytest.mark.parametrize("shape", [
    dict(B=16, Tq=1, T=8000, Hq=32, Hk=8, D=128, format=0),
    dict(B=16, Tq=1, T=8000, Hq=32, Hk=8, D=128, format=1),
    dict(B=32, Tq=16, T=777, Hq=16, Hk=2, D=128, N=4, P=6272, format=0),
    dict(B=32, Tq=16, T=777, Hq=16, Hk=2, D=128, N=4, P=6272, format=1),
    dict(B=4, Tq=3, T=900, Hq=8, Hk=2, D=100, N=1, P=5000, format=0),     # no 16-byte rows at all
], ids=str)
def test_a_workspace_is_sized_before_the_caches_exist(shape):
    """Caches given or not, at addresses of any alignment, lengths given or not:
    one size, and a call takes no more (16 sequences of 8000 plain keys were
    2129920 bytes without kv_len and 2795520 with it)."""
    first = size(desc(at=None, **shape))
    assert first > 0
    for at in (None, FAKE, FAKE + 4):
        for kv_len in (None, FAKE):
            a = desc(at=at, kv_len=kv_len, **shape)
            assert size(a) == first, (at, kv_len)
            if at is not None:
                assert _lib.load().mp3d_attention_cached(
                    ctypes.byref(a), FAKE, FAKE, FAKE, FAKE, first - 16, None) == _lib.MP3D_EWORKSPACE
