"""Attention over caches in blocks of 128 rows where the rows of codes start
anywhere, values that are not finite channel by channel, and caches past 2^32
bytes whose rows are read 16 bytes at a time."""
import pytest
import torch

import _caches as oracle
import _tokens as tk
import bwd_max_pool3d_amd as mp
from test_gpu_attention_cached import KINDS, make_cache, positions, run, spoil

pytestmark = pytest.mark.gpu

HALF = [torch.float16, torch.bfloat16]
SHAPES = [
    # B, N, Tq, Tk, P, Hq, Hk
    (20, 1, 1, 90, 300, 8, 1),             # 160 rows of a prefix, 8 of an own cache
    (4, 2, 20, 150, 70, 8, 2),             # 160 of a prefix, 80 of an own cache
    (2, 0, 70, 200, 0, 4, 2),              # 140 of an own cache: one chunk, nothing to join
    (2, 0, 33, 700, 0, 8, 2),              # 132, several chunks
    (9, 1, 1, 40, 129, 8, 1),              # 72
]


@pytest.mark.parametrize("dt", HALF, ids=tk.name_of)
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [72, 100, 101, 127])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("more", ["", "cap", "bias"])
def test_blocks_of_128_over_rows_that_start_anywhere(more, shape, D, fmt, dt):
    B, N, Tq, Tk, P, Hq, Hk = shape
    q = tk.randn((B, Tq, Hq, D), 1, dt)
    hk, own = make_cache(B, Tk, Hk, D, fmt, dt, 2)
    hp, prefix = make_cache(N, P, Hk, D, fmt, dt, 4) if N else (None, None)
    how = dict(kv_len=(Tk - torch.arange(B) * 3 % (Tk - Tq + 1)).int())
    for b in range(B):
        spoil(own, fmt, b, int(how["kv_len"][b]))
    if N:
        how["prefix_len"] = (P - 5 * torch.arange(N)).int()
        for n in range(N):
            spoil(prefix, fmt, n, int(how["prefix_len"][n]))
    if more == "cap":
        how["softcap"] = 3.0
    if more == "bias":
        how.update(positions(1 + D % 3, B, N, Tq, Tk, P, Hq, 6))
    got = run(q, own, prefix, fmt, how)
    want = oracle.attention(q, hk, hp, **how)
    for name in ("out", "lse"):
        tk.close(got[name], *want[name], name)


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("fmt", KINDS, ids=lambda f: f or "plain")
@pytest.mark.parametrize("D", [64, 72, 101, 128])
@pytest.mark.parametrize("Tq", [6, 70])
@pytest.mark.parametrize("P", [0, 40])
def test_channels_that_are_not_finite(P, Tq, D, fmt, dt):
    """Values that are not finite, of keys in the causal triangle: who sees the
    key is not finite in their channels, and all else is as without them."""
    B, Tk, Hq, Hk = 2, 130, 4, 2
    q = tk.randn((B, Tq, Hq, D), 11, dt)
    hk, own = make_cache(B, Tk, Hk, D, fmt, dt, 12)
    hp, prefix = make_cache(1, P, Hk, D, fmt, dt, 14) if P else (None, None)
    bad = torch.zeros(hk[1].shape, dtype=torch.bool)
    for b, back, h in ((0, 3, 1), (1, 1, 0), (1, Tq, 0)):  # seen by the last `back` tokens
        at = Tk - back
        if not fmt:
            own[1][b, at, h, D // 2], own[1][b, at, h, D - 1] = float("inf"), float("nan")
            bad[b, at, h, D // 2] = bad[b, at, h, D - 1] = True
        else:
            own[3][b, at, h, 1] = 255
            bad[b, at, h, 32:64] = True
            if fmt == "e4m3":
                own[2][b, at, h, D - 1] = 0x7F
                bad[b, at, h, D - 1] = True
    hk[1][bad] = 0
    got = run(q, own, prefix, fmt, {})
    want = oracle.attention(q, hk, hp)
    tk.close(got["lse"], *want["lse"], "lse")
    sees = torch.arange(Tk) <= torch.arange(Tq)[:, None] + Tk - Tq           # (Tq, Tk)
    hit = torch.einsum("tk,bkhd->bthd", sees.float(), bad.float()) > 0
    hit = hit.repeat_interleave(Hq // Hk, 2)
    out = got["out"].cpu()
    assert hit.any() and not torch.isfinite(out[hit]).any()
    value, tol = want["out"]
    zero = torch.zeros_like(value)
    tk.close(torch.where(hit, zero, out.double()), torch.where(hit, zero, value), tol, "out")


@pytest.mark.parametrize("Tq", [1, 40])
@pytest.mark.parametrize("fmt,dt", [("e4m3", torch.float16), ("e2m1", torch.float16),
                                    ("", torch.float16), ("", torch.float32)],
                         ids=["e4m3", "e2m1", "float16", "float32"])
def test_whole_rows_past_32_bits(fmt, dt, Tq):
    """Rows 2^24 - 128 bytes (plain: elements) apart, the largest stride with
    which they are read 16 (8) bytes at a time: the last ones lie more than 2^32
    bytes behind the first, and end inside a tile."""
    D, Hq, T, stride = 128, 2, 300 if fmt else 140, (1 << 24) - 128
    q = tk.randn((1, Tq, Hq, D), 21, dt)
    hk, small = make_cache(1, T, 1, D, fmt, dt, 22)
    far = []
    for i, t in enumerate(small):
        n = t.shape[3]
        big = torch.empty((T - 1) * stride + n, dtype=t.dtype, device="cuda")
        assert big.numel() * big.element_size() > 1 << 32
        far.append(big.as_strided((1, T, 1, n), (T * stride, stride, n, 1)))
        far[i].copy_(t)
    got, want = run(q, far, None, fmt, {}), oracle.attention(q, hk, None)
    for name in ("out", "lse"):
        tk.close(got[name], *want[name], name)
    near = run(q, small, None, fmt, {})
    for name in ("out", "lse"):
        assert torch.equal(got[name], near[name])
