"""Attention over caches at its ends, through the C ABI and the binding."""
import ctypes

import pytest
import torch

import _caches as oracle
import _tokens as tk
import bwd_max_pool3d_amd as mp
from bwd_max_pool3d_amd import _lib

pytestmark = pytest.mark.gpu

A3 = ctypes.c_int64 * 3


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("P", [0, 5, 20000])
def test_no_prefix_and_no_own_rows(P, dt):
    """prefix.B = 0 is no prefix whatever its T says: without rows of its own
    either, every query gets zeros (the launch had no workgroups)."""
    B, Tq, Hq, Hk, D = 3, 2, 4, 2, 64
    q = tk.randn((B, Tq, Hq, D), 1, dt).cuda()
    out, lse = torch.full_like(q, float("nan")), torch.full((B, Hq, Tq), float("nan"), device="cuda")
    a = _lib.AttentionCache()
    a.dtype = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[dt]
    a.B, a.Tq, a.Hq, a.Hk, a.D, a.causal, a.scale = B, Tq, Hq, Hk, D, 1, 1.0
    a.q_stride = A3(*q.stride()[:3])
    a.own.B, a.prefix.T = B, P
    n = ctypes.c_size_t()
    lib = _lib.load()
    assert lib.mp3d_attention_cached_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    ws = torch.empty(max(1, n.value), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    _lib.check(lib.mp3d_attention_cached(ctypes.byref(a), q.data_ptr(), out.data_ptr(),
                                         lse.data_ptr(), ws.data_ptr(), n.value, stream))
    assert torch.equal(out, torch.zeros_like(out))
    assert bool((lse == float("-inf")).all())


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("Tq", [1, 40])
@pytest.mark.parametrize("D", [7, 15, 47, 63, 101, 127])
def test_half_a_byte_that_is_no_channels(D, Tq, dt):
    """Heads of an odd width in 4 bits: the upper half of a row's last byte may
    hold anything (6 there, under the scale of a last group near the type's
    largest number, was an infinity, and the scores NaN)."""
    B, T, Hq, Hk, fmt = 2, 70, 4, 2, "e2m1"
    q = tk.randn((B, Tq, Hq, D), 1, dt)
    host, cache = [], []
    for i in range(2):
        x = tk.randn((B, T, Hk, D), 2 + i, dt)
        last = (D - 1) // 32 * 32
        x[..., last:] = 0                                  # codes 0, so that no score is large
        codes, scales = oracle.write(x, fmt)
        codes[..., -1] = 0x70
        scales[..., -1] = 142 if dt == torch.float16 else 254
        host.append(oracle.read(codes, scales, fmt, D, dt))
        assert torch.isfinite(host[i]).all()
        cache += [t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (codes, scales)]
    for got, want in zip(mp.mp3d_cache_read(cache, fmt, D, dt), host):
        assert torch.equal(got.cpu(), want)
    out, lse = mp.mp3d_attention_cached(q.cuda(), cache, format=fmt)
    want = oracle.attention(q, host)
    tk.close(out, *want["out"], "out")
    tk.close(lse, *want["lse"], "lse")
