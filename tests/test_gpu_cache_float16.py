"""Attention over caches in float16, where the weights' range ends at 2^-25."""
import math

import pytest
import torch

import _caches as oracle
import _tokens as tk
import bwd_max_pool3d_amd as mp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["", "e4m3"], ids=lambda f: f or "plain")
@pytest.mark.parametrize("B,Hq", [(1024, 1), (512, 128)], ids=["blocks of 16", "blocks of 128"])
def test_many_small_weights_behind_a_large_one(B, Hq, fmt):
    """2^20 keys of weight e^-18 = 2^-26 behind four of weight 1 (one for each
    wave of a workgroup, at its first tile's start), whose values are 0: what
    the many add up to is all of out."""
    dt, T, D = torch.float16, 1 << 20, 16
    k, v = torch.zeros((1, T, 1, D), dtype=dt), torch.ones((1, T, 1, D), dtype=dt)
    k[0, :, 0, 0] = -18.0                                  # (an e4m3 number times 2^-4)
    for key in (0, 32, 64, 96):
        k[0, key, 0, 0] = 0.0
        v[0, key] = 0.0
    parts = []
    for x in (k, v):
        if fmt:
            few = x[:, [0, 1]]
            codes, scales = oracle.write(few, fmt)
            assert torch.equal(oracle.read(codes, scales, fmt, D, dt), few)
            pick = (x[0, :, 0, 0] == few[0, 1, 0, 0]).long()
            parts += [codes[:, pick], scales[:, pick]]
        else:
            parts.append(x)
    # one cache in memory for all sequences
    cache = [p.cuda().expand(B, -1, -1, -1) for p in parts]
    q = torch.zeros((B, 1, Hq, D), dtype=dt, device="cuda")
    q[..., 0] = 1.0
    out, lse = mp.mp3d_attention_cached(q, cache, format=fmt or None, scale=1.0)
    total = 4.0 + (T - 4) * math.exp(-18.0)
    want = (T - 4) * math.exp(-18.0) / total
    # out and the weights are rounded once each; binary32 sums of a lane's T / 16
    # (blocks of 128: T / 2) weights and of as many products, 16 or 32 at a time
    lane, steps = (T // 16, T // 128) if Hq == 1 else (T // 2, T // 16)
    rel = 2 * tk.U[dt] + (lane + steps) * tk.E
    off = (out.double() - want).abs().max().item()
    assert off <= rel * want, (off / want, rel)
    off = (lse.double() - math.log(total)).abs().max().item()
    assert off <= (lane + 16) * tk.E, off
