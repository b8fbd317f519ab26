"""Attention over caches at its ends, through the C ABI and the binding."""
import ctypes

import pytest
import torch

import _tokens as tk
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
