"""Plain float64 forms of the token operators, on the CPU, with the error
bounds the kernels have to meet.

The bounds follow from how the results are formed, not from what was seen:
``U`` is a storage type's unit roundoff (half a unit in the last place over
the value), ``E`` = 2^-24 that of binary32.  Every result is rounded once to
the storage type (U |value|); operands of a second matrix product (weights
and their gradients) are rounded to it as well, and their errors pass
through the product with the absolute values of the other operand.
"""
from __future__ import annotations

import math

import torch

E = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# what a rounding to the type can add near 0 (half its smallest step)
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def name_of(dt):
    return str(dt).split(".")[-1]


def randn(shape, seed, dtype, scale=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + mean).to(dtype)


def close(got, want, tol, what=""):
    """|got - want| <= tol everywhere; infinities and NaN in the same places."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, "%s: shape %s" % (what, tuple(got.shape))
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), "%s: not finite elsewhere" % what
    assert torch.equal(torch.isnan(want), torch.isnan(got)), "%s: NaN elsewhere" % what
    rest = ~fine & ~torch.isnan(want)
    assert torch.equal(want[rest], got[rest]), "%s: infinities differ" % what
    off = torch.where(fine, (got - want).abs() - tol.expand_as(want), torch.zeros_like(want))
    if off.numel():
        worst = int(off.argmax())
        assert off.max() <= 0, "%s: off by %.3g, allowed %.3g, at %d (got %.9g, want %.9g)" % (
            what, float((got - want).abs().flatten()[worst]),
            float(tol.expand_as(want).flatten()[worst]), worst, float(got.flatten()[worst]),
            float(want.flatten()[worst]))


# ------------------------------------------------------------------ rope

def rope(x, inv_freq, pairs, pos, interleaved, sign=1.0):
    """(result, bound) for x (B, T, H, D), pos (3, B, T)."""
    dt = x.dtype
    x = x.double()
    P = sum(pairs)
    axis = [0] * pairs[0] + [1] * pairs[1] + [2] * pairs[2]
    y, size = x.clone(), torch.zeros_like(x)
    for i in range(P):
        a = sign * pos[axis[i]].double() * float(inv_freq[i].double())
        c, s = torch.cos(a)[..., None], torch.sin(a)[..., None]
        m, n = (2 * i, 2 * i + 1) if interleaved else (i, P + i)
        u, v = x[..., m].clone(), x[..., n].clone()
        y[..., m], y[..., n] = u * c - v * s, u * s + v * c
        size[..., m] = size[..., n] = u.abs() + v.abs()
    # sine and cosine within 2 E, two products and a sum
    return y, U[dt] * y.abs() + 5 * E * size + TINY[dt]


# ------------------------------------------------------------- attention

def spans(B, Tq, Tk, causal, kv_len, docs, prefix):
    """lo, hi (B, Tq): the keys each query sees (0, 0: none)."""
    lo, hi = torch.zeros(B, Tq, dtype=torch.long), torch.zeros(B, Tq, dtype=torch.long)
    for b in range(B):
        L = Tk if kv_len is None else max(0, min(Tk, int(kv_len[b])))
        for i in range(Tq):
            p = i + L - Tq
            s, e, n = 0, L, 0
            if docs is not None:
                off = [int(v) for v in docs[b]]
                here = [d for d in range(len(off) - 1) if off[d] <= p < off[d + 1]]
                if not here:
                    continue
                d = here[-1]
                s, e = max(off[d], 0), min(off[d + 1], L)
                if prefix is not None:
                    n = int(prefix[b][d])
            elif prefix is not None:
                n = int(prefix[b].reshape(-1)[0])
            if causal:
                e = min(e, max(p + 1, s + max(n, 0)))
            if e > s:
                lo[b, i], hi[b, i] = s, e
    return lo, hi


def attention(q, k, v, dout=None, *, scale=None, softcap=0.0, causal=False, kv_len=None,
              doc_offsets=None, prefix=None, slopes=None, pos_q=None, pos_k=None):
    """{name: (result, bound)} of out, lse and, with dout, dq, dk, dv."""
    dt = q.dtype
    u, tiny = U[dt], TINY[dt]
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    G = Hq // Hk
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    qd = q.double().permute(0, 2, 1, 3)
    kd = k.double().permute(0, 2, 1, 3).repeat_interleave(G, 1)
    vd = v.double().permute(0, 2, 1, 3).repeat_interleave(G, 1)
    raw = scale * (qd @ kd.transpose(2, 3))
    # a product's error, then the roundings of scale, cap and bias
    ds = (D + 4) * E * abs(scale) * (qd.abs() @ kd.abs().transpose(2, 3)) + 4 * E * raw.abs()
    s, slope = raw, None
    if softcap:
        t = torch.tanh(raw / softcap)
        s, slope = softcap * t, 1 - t * t
        ds = ds + 16 * E * softcap
    if slopes is not None:
        for a in range(slopes.shape[1]):
            gap = (pos_q[a].double()[:, :, None] - pos_k[a].double()[:, None, :]).abs()
            bias = slopes[:, a].double()[None, :, None, None] * gap[:, None]
            s = s - bias
            ds = ds + 8 * E * bias
    ds = ds + 4 * E * s.abs()
    lo, hi = spans(B, Tq, Tk, causal, kv_len, doc_offsets, prefix)
    j = torch.arange(Tk)
    see = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None]
    s = torch.where(see, s, torch.full_like(s, float("-inf")))
    ds = torch.where(see, ds, torch.zeros_like(ds))
    m = s.amax(-1, keepdim=True) if Tk else torch.full((B, Hq, Tq, 1), float("-inf")).double()
    p = torch.exp(s - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    lse = (m + torch.log(total))[..., 0]
    most = ds.amax(-1, keepdim=True) if Tk else torch.zeros_like(m)
    n = hi.max().item() + 16 if hi.numel() else 16
    dl = most[..., 0] + (math.sqrt(n) * 4 + 16) * E + 4 * E * torch.where(
        torch.isfinite(lse), lse.abs(), torch.zeros_like(lse))
    rel = 2 * (ds + most) + (math.sqrt(n) * 4 + 64) * E     # of a weight
    vis = lambda x: torch.where(see, x, torch.zeros_like(x))  # noqa: E731
    out = p @ vd
    o_tol = u * out.abs() + (p * (u + rel) + tiny) @ vd.abs() + tiny
    back = lambda x: x.permute(0, 2, 1, 3).contiguous()     # noqa: E731
    r = {"out": (back(out), back(o_tol)), "lse": (lse, dl)}
    if dout is None:
        return r
    do = dout.double().permute(0, 2, 1, 3)
    dp = do @ vd.transpose(2, 3)
    dp_size = do.abs() @ vd.abs().transpose(2, 3)
    delta = (do * out).sum(-1, keepdim=True)
    # delta is formed from the rounded out
    d_delta = (do.abs() * (2 * o_tol + D * E * out.abs())).sum(-1, keepdim=True)
    e = vis(p * (dp - delta))
    e_tol = vis(p * ((D + 8) * E * dp_size + d_delta) + e.abs() * (rel + u + 8 * E) + tiny)
    if slope is not None:
        # 1 - t^2 from a tanh within 4 E (plus the score's error)
        e_tol = e_tol * slope + e.abs() * (16 * E + 4 * ds / softcap)
        e = e * slope
    p_tol = vis(p * (u + rel) + tiny)
    dq, dq_t = scale * (e @ kd), abs(scale) * (e_tol @ kd.abs())
    dk, dk_t = scale * (e.transpose(2, 3) @ qd), abs(scale) * (e_tol.transpose(2, 3) @ qd.abs())
    dv, dv_t = p.transpose(2, 3) @ do, p_tol.transpose(2, 3) @ do.abs()
    # sums of up to Tq G products in binary32
    acc = (math.sqrt(max(Tq * G, Tk)) * 4 + 16) * E
    dq_t = dq_t + acc * abs(scale) * (e.abs() @ kd.abs())
    dk_t = dk_t + acc * abs(scale) * (e.abs().transpose(2, 3) @ qd.abs())
    dv_t = dv_t + acc * (p.transpose(2, 3) @ do.abs())
    share = lambda x: x.view(B, Hk, G, Tk, D).sum(2)        # noqa: E731
    dk, dk_t, dv, dv_t = share(dk), share(dk_t), share(dv), share(dv_t)
    for name, x, t in (("dq", dq, dq_t), ("dk", dk, dk_t), ("dv", dv, dv_t)):
        r[name] = (back(x), back(t + u * x.abs() + tiny))
    return r


# ------------------------------------------------------------ gated norm

def _norm(a, da, layer, eps):
    """n(a), 1 / deviation, and bounds of their errors (absolute and
    relative), from a's error da."""
    C = a.shape[-1]
    mean = a.mean(-1, keepdim=True) if layer else torch.zeros_like(a[..., :1])
    c = a - mean
    # sums of C terms: at most 16 in one thread, then a tree
    dm = (32 * E * a.abs().mean(-1, keepdim=True) + da.mean(-1, keepdim=True)) if layer else 0.0
    dc = da + dm + E * (a.abs() + mean.abs())
    var = (c * c).mean(-1, keepdim=True)
    dvar = 2 * (c.abs() * dc).mean(-1, keepdim=True) + 36 * E * var
    r = 1.0 / torch.sqrt(var + eps)
    rel = 0.75 * dvar / (var + eps) + 4 * E
    n = c * r
    return n, r, dc * r + n.abs() * rel, rel


def gated_norm(x, h, gate, post, pre, rs, layer, eps, post_norm=True, pre_norm=True, dy=None,
               dz=None, grads=False):
    """{name: (result, bound)}; gate is (G, C) or None."""
    dt = x.dtype
    u, tiny = U[dt], TINY[dt]
    C = x.shape[-1]
    one = torch.ones(C, dtype=torch.float64)
    x2 = x.double().reshape(-1, C)
    rows = x2.shape[0]
    g = one if gate is None else gate.double().repeat_interleave(rows // gate.shape[0], 0)
    wp = one if post is None else post.double()
    w = one if pre is None else pre.double()
    rs = float(torch.tensor(rs, dtype=torch.float32))
    r = {}
    y, dy_err = x2, torch.zeros_like(x2)
    if h is not None:
        h2 = h.double().reshape(-1, C)
        if post_norm:
            nh, rh, nh_err, rh_rel = _norm(h2, torch.zeros_like(h2), layer, eps)
        else:
            nh, rh, nh_err, rh_rel = h2, None, torch.zeros_like(h2), None
        f = rs * g * wp
        y = x2 + f * nh
        dy_err = f.abs() * nh_err + 8 * E * (f * nh).abs() + 2 * E * y.abs()
        r["y"] = (y, dy_err + u * y.abs() + tiny)
    if pre_norm:
        ny, ry, ny_err, ry_rel = _norm(y, dy_err, layer, eps)
        z = w * ny
        r["z"] = (z, w.abs() * ny_err + u * z.abs() + 4 * E * z.abs() + tiny)
    if not grads:
        return {k: (a.view(x.shape), b.view(x.shape)) for k, (a, b) in r.items()}

    def back(d, d_err, n, n_err, rr, rel):
        """gradient of n(a) at a, from d at n: value and error."""
        m1 = (d * n).mean(-1, keepdim=True)
        e1 = (d_err * n.abs() + d.abs() * n_err).mean(-1, keepdim=True) + 40 * E * (
            d * n).abs().mean(-1, keepdim=True)
        m2 = d.mean(-1, keepdim=True) if layer else torch.zeros_like(m1)
        e2 = (d_err.mean(-1, keepdim=True) + 40 * E * d.abs().mean(-1, keepdim=True)) if layer \
            else 0.0
        val = (d - m2 - n * m1) * rr
        size = (d.abs() + m2.abs() + (n * m1).abs()) * rr
        return val, (d_err + e2 + n.abs() * e1 + n_err * m1.abs()) * rr + size * (rel + 8 * E)

    dx = torch.zeros_like(x2) if dy is None else dy.double().reshape(-1, C)
    dx_err = torch.zeros_like(x2)
    sums = lambda t, e: (t.sum(0), e.sum(0) + (math.sqrt(rows) * 4 + 32) * E * t.abs().sum(0))  # noqa: E731
    if pre_norm:
        d = dz.double().reshape(-1, C)
        val, err = back(w * d, 2 * E * (w * d).abs(), ny, ny_err, ry, ry_rel)
        dx = dx + val
        dx_err = err + 2 * E * dx.abs()
        if pre is not None:
            r["dpre"] = sums(d * ny, d.abs() * ny_err)
    r["dx"] = (dx, dx_err + u * dx.abs() + tiny)
    if h is not None:
        d, d_err = f * dx, f.abs() * dx_err + 4 * E * (f * dx).abs()
        dh, dh_err = back(d, d_err, nh, nh_err, rh, rh_rel) if post_norm else (d, d_err)
        r["dh"] = (dh, dh_err + u * dh.abs() + tiny)
        t = rs * dx * nh
        t_err = abs(rs) * (dx.abs() * nh_err + dx_err * nh.abs()) + 4 * E * t.abs()
        if post is not None:
            r["dpost"] = sums(t * g, t_err * g.abs())
        if gate is not None:
            a = (t * wp).view(gate.shape[0], -1, C)
            b = (t_err * wp.abs()).view(gate.shape[0], -1, C)
            n = a.shape[1]
            r["dgate"] = (a.sum(1), b.sum(1) + (math.sqrt(n) * 4 + 32) * E * a.abs().sum(1))
    return {k: (a.view(x.shape), b.view(x.shape)) if a.shape == x2.shape and k in
            ("y", "z", "dx", "dh") else (a, b) for k, (a, b) in r.items()}
