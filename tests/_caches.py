"""Plain forms, on the CPU and in float64, of the caches in 8 and 4 bits and of
attention over caches; attention's bounds are those of _tokens.

A code and a scale byte are whole numbers with one right answer, and a value
read back is one rounding of an exact product, so these are compared bit for
bit.
"""
from __future__ import annotations

import math

import torch

import _tokens as tk

FORMATS = ["e4m3", "e2m1"]
LARGEST = {torch.float32: 3.4028234663852886e38, torch.float16: 65504.0,
           torch.bfloat16: 3.3895313892515355e38}


def magnitudes(fmt):
    """The format's numbers >= 0, in the order of their codes."""
    if fmt == "e2m1":
        return [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    out = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        out += [(8 + m) * 2.0 ** (e - 10) for m in range(8)]
    return out[:-1]                                    # the last code is NaN


def widths(fmt, D):
    return (D if fmt == "e4m3" else (D + 1) // 2), (D + 31) // 32


def write(x, fmt):
    """(codes, scales) of x (..., D), uint8."""
    mags = magnitudes(fmt)
    D = x.shape[-1]
    width, groups = widths(fmt, D)
    g = torch.zeros(x.shape[:-1] + (groups * 32,), dtype=torch.float64)
    g[..., :D] = x.double()
    g = g.unflatten(-1, (groups, 32))
    a = g.abs().amax(-1)
    bad = ~torch.isfinite(g).all(-1)
    a = torch.where(bad, torch.ones_like(a), a)
    s = torch.full(a.shape, -126.0, dtype=torch.float64)
    for e in range(-126, 128):
        s = torch.where(a > mags[-1] * 2.0 ** e, torch.full_like(s, e + 1.0), s)
    unit = torch.exp2(s)[..., None]
    r = torch.where(bad[..., None], torch.zeros_like(g), g.abs() / unit)
    m = torch.tensor(mags, dtype=torch.float64)
    # the nearest number; between two, the one of the even code
    code = torch.zeros(r.shape, dtype=torch.long)
    for i in range(1, len(mags)):
        mid = (mags[i] + mags[i - 1]) / 2
        up = (r > mid) | ((r == mid) & (i % 2 == 0))
        code = torch.where(up, torch.full_like(code, i), code)
    # the largest within the type
    top = (m * unit <= LARGEST[x.dtype]).sum(-1, keepdim=True) - 1
    code = torch.minimum(code, top)
    sign = torch.signbit(g) & ~bad[..., None]
    bits = 8 if fmt == "e4m3" else 4
    code = (code + (sign.long() << (bits - 1))).flatten(-2)
    scales = torch.where(bad, torch.full_like(s, 255.0), s + 127).to(torch.uint8)
    if fmt == "e2m1":
        code = code[..., 0::2] + 16 * code[..., 1::2]
    return code[..., :width].to(torch.uint8), scales


def read(codes, scales, fmt, D, dtype):
    """The values of codes and scales, in dtype."""
    mags = torch.tensor(magnitudes(fmt) + ([float("nan")] if fmt == "e4m3" else []),
                        dtype=torch.float64)
    c = codes.long()
    if fmt == "e2m1":
        c = torch.stack((c % 16, c // 16), -1).flatten(-2)[..., :D]
    half = len(mags)
    x = mags[c % half] * torch.where(c >= half, -1.0, 1.0).double()
    s = scales.long()
    unit = torch.exp2(s.double() - 127)
    unit = torch.where(s == 255, torch.full_like(unit, float("nan")), unit)
    x = x * unit.repeat_interleave(32, -1)[..., :D]
    return x.to(dtype) if dtype != torch.bfloat16 else to_bf16(x)


def to_bf16(x):
    """float64 to bfloat16 with one rounding (every value here has at most 4
    significant bits: float32 holds it, or is below or above its range)."""
    return x.float().to(torch.bfloat16)


def attention(q, own, prefix=None, *, scale=None, softcap=0.0, causal=True, kv_len=None,
              prefix_len=None, slopes=None, pos_q=None, pos_k=None, pos_prefix=None):
    """{name: (result, bound)}; own and prefix are (k, v) of q's type."""
    B, Tq, Hq, D = q.shape
    out, lse = [], []
    for b in range(B):
        L = own[0].shape[1] if kv_len is None else max(0, min(int(kv_len[b]), own[0].shape[1]))
        k, v = own[0][b:b + 1, :L], own[1][b:b + 1, :L]
        P, how = 0, {}
        if prefix is not None:
            n = b // (B // prefix[0].shape[0])
            P = prefix[0].shape[1]
            if prefix_len is not None:
                P = max(0, min(int(prefix_len[n]), P))
            k = torch.cat((prefix[0][n:n + 1, :P], k), 1)
            v = torch.cat((prefix[1][n:n + 1, :P], v), 1)
        if slopes is not None:
            pk = pos_k[:, b:b + 1, :L]
            if prefix is not None:
                pk = torch.cat((pos_prefix[:, n:n + 1, :P], pk), 2)
            how = dict(slopes=slopes, pos_q=pos_q[:, b:b + 1], pos_k=pk)
        r = tk.attention(q[b:b + 1], k, v, scale=scale, softcap=softcap, causal=causal,
                         prefix=torch.tensor([[P]]) if causal else None, **how)
        out.append(r["out"])
        lse.append(r["lse"])
    join = lambda x: tuple(torch.cat([y[i] for y in x]) for i in range(2))  # noqa: E731
    value, tol = join(out)
    lv, lt = join(lse)
    # the chunks' sums, joined: a product and a sum for each, in binary32
    size = math.sqrt(64) * 4 * tk.E
    return {"out": (value, tol + size * value.abs()), "lse": (lv, lt + size)}
