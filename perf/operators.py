"""The token operators that follow a 3-D max pool, as cases to measure: rotary
positions over the volume's axes, attention over its tokens, and the norm
that joins a block's output to the residual stream.

Each case is one pass through one operator as a training step or a decoding
loop makes it.  ``run`` computes it in plain torch (elementary operations in
float32, rounded once at the end), or, where the module's ``own`` is true,
by this package's kernels; ``exact`` computes it from the definition in
float64.

Definitions (B sequences of T tokens, heads of D channels):

  rope       pair i of a head's first 2P channels turns by the angle
             position[axis(i)] * inv_freq[i]; axis(i) by ``sections``.  The
             backward turns by the negative angle.
  attention  s = scale q.k, then cap tanh(s / cap), then minus
             sum_a slope[h, a] |pos_q[a, i] - pos_k[a, j]|.  Query i stands
             at p = i + kv_len - Tq and sees the keys [lo, hi) of its
             document, up to max(p + 1, start + prefix) if causal.  A query
             that sees nothing gives 0 (and a log-sum-exp of -infinity).
  norm       y = x + residual_scale gate (post_weight n(h)),
             z = pre_weight n(y), n the RMS or the layer norm.
"""
import math

import torch

own = False

_TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
_BYTES = {"float32": 4, "float16": 2, "bfloat16": 2}
_EPS = 1e-6


def _rope_case(name, dtype, pass_, B, grid, Hq, Hk, D, pairs, interleaved=False, positions=False):
    return {"name": name, "op": "rope", "dtype": dtype, "pass": pass_, "B": B, "gd": grid[0],
            "gh": grid[1], "gw": grid[2], "Hq": Hq, "Hk": Hk, "D": D, "pd": pairs[0],
            "ph": pairs[1], "pw": pairs[2], "interleaved": interleaved, "positions": positions}


def _attn_case(name, dtype, pass_, B, Tq, Tk, Hq, Hk, D, cap=0.0, causal=False, docs=0,
               prefix=False, axes=0, ragged=False, head_major=False):
    return {"name": name, "op": "attention", "dtype": dtype, "pass": pass_, "B": B, "Tq": Tq,
            "Tk": Tk, "Hq": Hq, "Hk": Hk, "D": D, "cap": cap, "causal": causal, "docs": docs,
            "prefix": prefix, "axes": axes, "ragged": ragged, "head_major": head_major}


def _norm_case(name, dtype, pass_, B, T, C, kind, gate="batch"):
    return {"name": name, "op": "norm", "dtype": dtype, "pass": pass_, "B": B, "T": T, "C": C,
            "kind": kind, "gate": gate}


def listed():
    return [
        # one new token of each of 32 sequences: latency
        _rope_case("rope_decode", "bfloat16", "forward", 32, (1, 1, 1), 16, 4, 128, (16, 24, 24),
                   positions=True),
        # the tokens of four (8, 56, 56) volumes, which a 2x2x2 pool of (16, 112, 112) leaves
        _rope_case("rope_volume", "bfloat16", "forward", 4, (8, 56, 56), 16, 4, 128, (16, 24, 24)),
        # gradients of 32 pooled (5, 7, 7) volumes, adjacent pairs, some channels not turned
        _rope_case("rope_grad_f32", "float32", "backward", 32, (5, 7, 7), 12, 12, 80, (8, 12, 12),
                   interleaved=True, positions=True),
        # a long prompt, the tokens of one (15, 27, 27) volume, with capped scores
        _attn_case("attn_prompt_cap", "bfloat16", "forward", 1, 10935, 10935, 16, 4, 128, cap=50.0,
                   causal=True),
        # a training step over clips packed into one row, near cells favoured on all three axes
        _attn_case("attn_docs_train", "bfloat16", "train", 1, 8192, 8192, 16, 16, 64, docs=9,
                   axes=3),
        # a training step in which a prompt sees itself both ways; odd length, shared heads
        _attn_case("attn_prefix_train", "float16", "train", 2, 2047, 2047, 16, 2, 128, causal=True,
                   prefix=True),
        # many small pooled volumes in float32
        _attn_case("attn_small_f32", "float32", "train", 32, 245, 245, 4, 4, 64, axes=3),
        # decoding with long caches of different lengths: the caches are read once
        _attn_case("attn_decode_long", "bfloat16", "forward", 16, 1, 32768, 32, 8, 128, causal=True,
                   ragged=True, head_major=True),
        # decoding at the start of one sequence: latency
        _attn_case("attn_decode_short", "float16", "forward", 1, 1, 777, 16, 4, 128, cap=30.0,
                   causal=True, axes=1),
        # one decoding step of 32 sequences: latency
        _norm_case("norm_decode", "bfloat16", "forward", 32, 1, 2048, "rms", gate="channel"),
        # a training step over four (15, 27, 27) volumes
        _norm_case("norm_train", "bfloat16", "train", 4, 10935, 1024, "rms"),
        # a training step over 32 pooled (5, 7, 7) volumes, an odd width
        _norm_case("norm_layer_f32", "float32", "train", 32, 245, 1001, "layer"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "attention", "attention", "norm"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
    if op == "rope":
        D = 2 * rng.randint(8, 64)
        pd, ph, pw = (rng.randint(0, D // 6) for _ in range(3))
        pw = max(pw, 1)
        Hk = rng.choice((1, 2, 4, 8))
        grid = (_log_int(rng, 1, 16), _log_int(rng, 1, 56), _log_int(rng, 1, 56))
        B = _log_int(rng, 1, max(1, min(32, 40000 // (grid[0] * grid[1] * grid[2]))))
        return _rope_case("", dtype, rng.choice(("forward", "backward")), B, grid,
                          Hk * rng.choice((1, 2, 3, 4)) if Hk < 8 else 16, Hk, D, (pd, ph, pw),
                          interleaved=rng.random() < 0.5, positions=rng.random() < 0.5)
    if op == "norm":
        C = _log_int(rng, 8, 4096)
        B = _log_int(rng, 1, 32)
        T = _log_int(rng, 1, max(1, min(10935, 40_000_000 // (B * C))))
        return _norm_case("", dtype, rng.choice(("forward", "train")), B, T, C,
                          rng.choice(("rms", "layer")), rng.choice(("batch", "channel", "none")))
    Hk = rng.choice((1, 2, 4, 8))
    Hq = Hk * rng.choice((1, 2, 4)) if Hk < 8 else rng.choice((8, 16, 32))
    D = rng.choice((32, 64, 72, 96, 128, 128))
    cap = rng.choice((0.0, 0.0, 20.0, 50.0))
    if rng.random() < 0.35:                      # decoding, one to four new tokens
        Tk = _log_int(rng, 64, 32768)
        B = _log_int(rng, 1, max(1, min(32, 4_000_000 // (Tk * Hk))))
        return _attn_case("", dtype, "forward", B, rng.choice((1, 1, 1, 2, 4)), Tk, Hq, Hk, D,
                          cap=cap, causal=True, axes=rng.choice((0, 0, 1)), ragged=True,
                          head_major=rng.random() < 0.5)
    T = _log_int(rng, 16, 6000)
    B = _log_int(rng, 1, max(1, min(16, 400_000_000 // (T * T * Hq))))
    docs = rng.choice((0, 0, rng.randint(2, 8)))
    causal = rng.random() < 0.6
    return _attn_case("", dtype, rng.choice(("forward", "train", "train")), B, T, T, Hq, Hk, D,
                      cap=cap, causal=causal, docs=docs if T >= 64 else 0,
                      prefix=causal and rng.random() < 0.4, axes=rng.choice((0, 0, 1, 3)))


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Host lists a case implies: (kv_len per sequence, document starts,
    prefix per document)."""
    B, Tk, docs = case["B"], case["Tk"], case["docs"]
    kv = [Tk - (b * (3 * Tk // 4)) // B for b in range(B)] if case["ragged"] else [Tk] * B
    kv = [max(n, 1) for n in kv]
    if docs:
        # lengths in the ratio 1 : 2 : 3 ... in a mixed order, the last tokens in no document
        w = [1 + (7 * d + 3) % docs for d in range(docs)]
        used = Tk - Tk // 50
        off = [0]
        for d in range(docs):
            off.append(off[-1] + used * w[d] // sum(w))
    else:
        off = [0, Tk]
    pre = [(off[d + 1] - off[d]) // 3 if case["prefix"] else 0 for d in range(len(off) - 1)]
    return kv, off, pre


def _rand(shape, gen, dtype, scale=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale + mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]
    dev = "cuda"
    B = case["B"]
    st = {"case": case}
    if case["op"] == "rope":
        T = case["gd"] * case["gh"] * case["gw"]
        P = case["pd"] + case["ph"] + case["pw"]
        # q and k as the two ends of one projection's output
        qk = _rand((B, T, case["Hq"] + case["Hk"], case["D"]), gen, dt)
        st["q"], st["k"] = qk[:, :, :case["Hq"]], qk[:, :, case["Hq"]:]
        st["inv_freq"] = torch.tensor([10000.0 ** (-i / P) for i in range(P)], device=dev)
        if case["positions"]:
            t = torch.arange(T, device=dev)
            cell = torch.stack((t // (case["gh"] * case["gw"]), t // case["gw"] % case["gh"],
                                t % case["gw"]))
            start = torch.randint(0, 4096, (3, B, 1), generator=gen, device=dev)
            st["positions"] = (cell[:, None, :] + start).to(torch.int32).contiguous()
        else:
            st["positions"] = None
        return st
    if case["op"] == "norm":
        shape = (B, case["T"], case["C"])
        st["x"], st["h"] = _rand(shape, gen, dt), _rand(shape, gen, dt, 2.0, 0.25)
        st["post"] = _rand((case["C"],), gen, dt, 0.1, 1.0)
        st["pre"] = _rand((case["C"],), gen, dt, 0.1, 1.0)
        rows = {"batch": B, "channel": 1, "none": 0}[case["gate"]]
        st["gate"] = _rand((rows, case["C"]), gen, dt, 0.5) if rows else None
        if case["pass"] == "train":
            st["dy"], st["dz"] = _rand(shape, gen, dt), _rand(shape, gen, dt)
        return st
    Hq, Hk, D, Tq, Tk = (case[n] for n in ("Hq", "Hk", "D", "Tq", "Tk"))
    kv, off, pre = _lengths(case)
    if case["head_major"]:                       # a cache laid out (B, H, T, D)
        st["q"] = _rand((B, Tq, Hq, D), gen, dt)
        st["k"] = _rand((B, Hk, Tk, D), gen, dt).transpose(1, 2)
        st["v"] = _rand((B, Hk, Tk, D), gen, dt).transpose(1, 2)
    else:
        st["q"], st["k"], st["v"] = (_rand((B, T, H, D), gen, dt)
                                     for T, H in ((Tq, Hq), (Tk, Hk), (Tk, Hk)))
    st["kv_len"] = (torch.tensor(kv, dtype=torch.int32, device=dev) if case["ragged"] else None)
    st["docs"] = (torch.tensor([off] * B, dtype=torch.int32, device=dev) if case["docs"] else None)
    st["prefix"] = (torch.tensor([pre] * B, dtype=torch.int32, device=dev)
                    if case["prefix"] else None)
    A = case["axes"]
    if A:
        # positions in a volume 27 cells high and wide (one axis: the token's number)
        t = torch.arange(Tk, device=dev, dtype=torch.int32)
        cell = torch.stack((t // 729, t // 27 % 27, t % 27)) if A == 3 else t[None]
        st["pos_k"] = cell[:, None, :].expand(A, B, Tk).contiguous()
        at = (torch.tensor(kv, device=dev)[:, None] - Tq + torch.arange(Tq, device=dev)).clamp(min=0)
        st["pos_q"] = st["pos_k"].gather(2, at[None].expand(A, B, Tq)).contiguous()
        st["slopes"] = (torch.rand((Hq, A), generator=gen, device=dev) + 0.5) * (
            2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq))[:, None]
    else:
        st["pos_q"] = st["pos_k"] = st["slopes"] = None
    if case["pass"] == "train":
        st["dout"] = _rand((B, Tq, Hq, D), gen, dt)
    return st


# ----------------------------------------------------------------- passes

def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["op"]](state, case)


def _own_rope(st, c):
    import bwd_max_pool3d_amd as mp
    call = mp.mp3d_rope_backward if c["pass"] == "backward" else mp.mp3d_rope_forward
    return call(st["q"], st["k"], st["inv_freq"], (c["pd"], c["ph"], c["pw"]),
                positions=st["positions"], grid=(c["gd"], c["gh"], c["gw"]) if st["positions"] is None
                else None, interleaved=c["interleaved"])


def _own_attention(st, c):
    import bwd_max_pool3d_amd as mp
    how = dict(softcap=c["cap"], causal=c["causal"], kv_len=st["kv_len"], doc_offsets=st["docs"],
               prefix=st["prefix"], slopes=st["slopes"], pos_q=st["pos_q"], pos_k=st["pos_k"])
    out, lse = mp.mp3d_attention_forward(st["q"], st["k"], st["v"], **how)
    if c["pass"] == "forward":
        return out, lse
    return (out, lse) + mp.mp3d_attention_backward(st["dout"], st["q"], st["k"], st["v"], out, lse,
                                                   **how)


def _own_norm(st, c):
    import bwd_max_pool3d_amd as mp
    how = dict(gate=st["gate"], post_weight=st["post"], pre_weight=st["pre"], residual_scale=0.5,
               norm=c["kind"], eps=_EPS)
    y, z, stats = mp.mp3d_gated_norm_forward(st["x"], st["h"], **how)
    if c["pass"] == "forward":
        return y, z
    g = mp.mp3d_gated_norm_backward(st["dy"], st["dz"], st["x"], st["h"], stats, **how)
    return (y, z) + tuple(t for t in g if t is not None)


_own = {"rope": _own_rope, "attention": _own_attention, "norm": _own_norm}


def _plain_rope(st, c):
    q, k, f = st["q"], st["k"], st["inv_freq"]
    B, T, Hq, D = q.shape
    P = f.numel()
    if st["positions"] is None:
        t = torch.arange(T, device=q.device)
        pos = torch.stack((t // (c["gh"] * c["gw"]), t // c["gw"] % c["gh"], t % c["gw"]))[:, None]
    else:
        pos = st["positions"]
    axis = torch.repeat_interleave(torch.arange(3, device=q.device),
                                   torch.tensor((c["pd"], c["ph"], c["pw"]), device=q.device),
                                   output_size=P)
    angle = pos.float()[axis].permute(1, 2, 0) * f                  # (B or 1, T, P)
    cos, sin = angle.cos()[:, :, None], angle.sin()[:, :, None]
    if c["pass"] == "backward":
        sin = -sin
    x = torch.cat((q, k), 2).float()
    if c["interleaved"]:
        u, v = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
    else:
        u, v = x[..., :P], x[..., P:2 * P]
    a, b = u * cos - v * sin, u * sin + v * cos
    turned = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    out = torch.cat((turned, x[..., 2 * P:]), -1).to(q.dtype)
    return out[:, :, :Hq].contiguous(), out[:, :, Hq:].contiguous()


def _visible(st, c, device):
    """(B, Tq, Tk) truth values: which keys each query sees."""
    B, Tq, Tk = c["B"], c["Tq"], c["Tk"]
    length = (torch.full((B, 1), Tk, device=device) if st["kv_len"] is None
              else st["kv_len"][:, None].long())
    p = torch.arange(Tq, device=device) + length - Tq
    if st["docs"] is None:
        start, end = torch.zeros_like(p), length.expand_as(p)
        pre = torch.zeros_like(p) if st["prefix"] is None else st["prefix"][:, :1].expand_as(p)
    else:
        off = st["docs"].long()
        d = torch.searchsorted(off, p, right=True) - 1
        inside = (d >= 0) & (d < off.shape[1] - 1)
        d = d.clamp(0, off.shape[1] - 2)
        start = off.gather(1, d)
        end = torch.where(inside, torch.minimum(off.gather(1, d + 1), length), start)
        pre = torch.zeros_like(p) if st["prefix"] is None else st["prefix"].gather(1, d)
    if c["causal"]:
        end = torch.minimum(end, torch.maximum(p + 1, start + pre))
    j = torch.arange(Tk, device=device)
    return (j >= start[..., None]) & (j < end[..., None])


def _plain_attention(st, c):
    q, k, v = st["q"], st["k"], st["v"]
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    G, scale = Hq // Hk, 1.0 / math.sqrt(D)
    qf = q.float().permute(0, 2, 1, 3).reshape(B, Hk, G * Tq, D)
    kf = k.float().permute(0, 2, 1, 3).contiguous()
    vf = v.float().permute(0, 2, 1, 3).contiguous()
    s = (qf * scale) @ kf.transpose(2, 3).contiguous()
    slope = None
    if c["cap"]:
        t = torch.tanh(s / c["cap"])
        if c["pass"] == "train":
            slope = 1 - t * t
        s = c["cap"] * t
    s = s.view(B, Hk, G, Tq, Tk)
    if st["slopes"] is not None:
        far = (st["pos_q"][..., :, None] - st["pos_k"][..., None, :]).abs().float()
        bias = st["slopes"] @ far.view(far.shape[0], -1)            # (Hq, B Tq Tk)
        s = s - bias.view(Hk, G, B, Tq, Tk).permute(2, 0, 1, 3, 4)
    s = s.masked_fill(~_visible(st, c, q.device)[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.masked_fill(m == float("-inf"), 0.0))
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).view(B, Hq, Tq)
    p = (p / total.masked_fill(total == 0, 1.0)).view(B, Hk, G * Tq, Tk)
    o = p @ vf
    out = o.view(B, Hq, Tq, D).permute(0, 2, 1, 3).to(q.dtype).contiguous()
    if c["pass"] == "forward":
        return out, lse
    do = st["dout"].float().permute(0, 2, 1, 3).reshape(B, Hk, G * Tq, D)
    dv = p.transpose(2, 3).contiguous() @ do
    ds = p * (do @ vf.transpose(2, 3).contiguous() - (do * o).sum(-1, keepdim=True))
    if slope is not None:
        ds = ds * slope
    dq = (ds @ kf) * scale
    dk = ds.transpose(2, 3).contiguous() @ (qf * scale)
    return (out, lse, dq.view(B, Hq, Tq, D).permute(0, 2, 1, 3).to(q.dtype).contiguous(),
            dk.permute(0, 2, 1, 3).to(q.dtype).contiguous(),
            dv.permute(0, 2, 1, 3).to(q.dtype).contiguous())


def _normed(a, kind):
    """n(a) and the reciprocal deviation, over the last axis."""
    if kind == "layer":
        a = a - a.mean(-1, keepdim=True)
    r = torch.rsqrt((a * a).mean(-1, keepdim=True) + _EPS)
    return a * r, r


def _norm_grad(d, n, r, kind):
    """The gradient at a of n(a), from the gradient d at n."""
    g = d - n * (d * n).mean(-1, keepdim=True)
    if kind == "layer":
        g = g - d.mean(-1, keepdim=True)
    return g * r


def _plain_norm(st, c):
    x, h, post, pre = (st[n].float() for n in ("x", "h", "post", "pre"))
    gate = None if st["gate"] is None else st["gate"].float()[:, None, :]
    nh, rh = _normed(h, c["kind"])
    w = 0.5 * post if gate is None else 0.5 * post * gate
    y = x + nh * w
    ny, ry = _normed(y, c["kind"])
    dt = st["x"].dtype
    first = (y.to(dt), (ny * pre).to(dt))
    if c["pass"] == "forward":
        return first
    dy, dz = st["dy"].float(), st["dz"].float()
    dx = dy + _norm_grad(dz * pre, ny, ry, c["kind"])
    t = dx * nh * 0.5
    dgate = None
    if gate is not None:
        dgate = (t * post).sum(1) if gate.shape[0] > 1 or c["gate"] == "batch" else (t * post).sum(
            (0, 1))[None]
        t = t * gate
    grads = (dx.to(dt), _norm_grad(dx * w, nh, rh, c["kind"]).to(dt), dgate, t.sum((0, 1)),
             (dz * ny).sum((0, 1)))
    return first + tuple(g for g in grads if g is not None)


_plain = {"rope": _plain_rope, "attention": _plain_attention, "norm": _plain_norm}


# -------------------------------------------------------------- definitions

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "attention": _exact_attention, "norm": _exact_norm}[case["op"]](
        st, case)


def _exact_rope(st, c):
    sizes = (c["pd"], c["ph"], c["pw"])
    T = c["gd"] * c["gh"] * c["gw"]
    sign = -1.0 if c["pass"] == "backward" else 1.0
    outs = []
    for name in ("q", "k"):
        x = st[name].double()
        y = x.clone()
        i = 0
        P = sum(sizes)
        for axis, n in enumerate(sizes):
            for _ in range(n):
                if st["positions"] is not None:
                    pos = st["positions"][axis].double()
                else:
                    t = torch.arange(T, device=x.device)
                    d, r = t // (c["gh"] * c["gw"]), t % (c["gh"] * c["gw"])
                    pos = (d, r // c["gw"], r % c["gw"])[axis].double().expand(c["B"], T)
                w = pos * float(st["inv_freq"][i].double()) * sign
                one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, P + i)
                z = torch.complex(x[..., one], x[..., two]) * torch.polar(
                    torch.ones_like(w), w)[:, :, None]
                y[..., one], y[..., two] = z.real, z.imag
                i += 1
        outs.append(y)
    return tuple(outs)


def _exact_attention(st, c):
    B, Tq, Hq, D = st["q"].shape
    Tk, Hk = c["Tk"], c["Hk"]
    kv, off, pre = _lengths(c)
    dev, f64 = st["q"].device, torch.float64
    train = c["pass"] == "train"
    out = torch.zeros(B, Tq, Hq, D, dtype=f64, device=dev)
    lse = torch.full((B, Hq, Tq), float("-inf"), dtype=f64, device=dev)
    dq = torch.zeros_like(out)
    dk = torch.zeros(B, Tk, Hk, D, dtype=f64, device=dev)
    dv = torch.zeros_like(dk)
    for b in range(B):
        first = kv[b] - Tq
        # each document on its own: its queries against its keys, one head at a time
        for lo, hi, n in zip(off, off[1:], pre):
            hi = min(hi, kv[b])
            i0, i1 = max(0, lo - first), max(0, min(Tq, hi - first))
            if i0 >= i1 or lo >= hi:
                continue
            i, j = torch.arange(i0, i1, device=dev), torch.arange(lo, hi, device=dev)
            hide = None
            if c["causal"]:
                hide = (j[None] > i[:, None] + first) & (j[None] >= lo + n)
            for h in range(Hq):
                g = h // (Hq // Hk)
                q, k, v = (st["q"][b, i0:i1, h].double(), st["k"][b, lo:hi, g].double(),
                           st["v"][b, lo:hi, g].double())
                raw = torch.matmul(q, k.t()) / math.sqrt(D)
                s = raw if not c["cap"] else c["cap"] * torch.tanh(raw / c["cap"])
                chain = 1.0 if not c["cap"] else 1.0 - (s / c["cap"]) ** 2
                if st["slopes"] is not None:
                    for a in range(st["slopes"].shape[1]):
                        gap = (st["pos_q"][a, b, i0:i1].double()[:, None]
                               - st["pos_k"][a, b, lo:hi].double()[None])
                        s = s - float(st["slopes"][h, a].double()) * gap.abs()
                if hide is not None:
                    s = torch.where(hide, torch.full_like(s, float("-inf")), s)
                lse[b, h, i0:i1] = torch.logsumexp(s, 1)
                w = torch.softmax(s, 1)
                out[b, i0:i1, h] = torch.matmul(w, v)
                if train:
                    do = st["dout"][b, i0:i1, h].double()
                    dv[b, lo:hi, g] += torch.matmul(w.t(), do)
                    back = torch.matmul(do, v.t())
                    back = w * (back - (w * back).sum(1, keepdim=True)) * chain / math.sqrt(D)
                    dq[b, i0:i1, h] = torch.matmul(back, k)
                    dk[b, lo:hi, g] += torch.matmul(back.t(), q)
    return (out, lse, dq, dk, dv) if train else (out, lse)


def _exact_norm(st, c):
    leaves = {n: st[n].double().requires_grad_(c["pass"] == "train")
              for n in ("x", "h", "gate", "post", "pre") if st[n] is not None}

    def norm(a):
        if c["kind"] == "layer":
            return (a - a.mean(-1, keepdim=True)) / torch.sqrt(
                a.var(-1, unbiased=False, keepdim=True) + _EPS)
        return a / torch.sqrt(a.pow(2).mean(-1, keepdim=True) + _EPS)

    u = norm(leaves["h"]) * leaves["post"] * 0.5
    if "gate" in leaves:
        u = u * leaves["gate"].unsqueeze(1)
    y = leaves["x"] + u
    z = norm(y) * leaves["pre"]
    if c["pass"] == "forward":
        return y, z
    loss = (y * st["dy"].double()).sum() + (z * st["dz"].double()).sum()
    order = [n for n in ("x", "h", "gate", "post", "pre") if n in leaves]
    return (y.detach(), z.detach()) + torch.autograd.grad(loss, [leaves[n] for n in order])


# --------------------------------------------------------------------- work

def work(case):
    c, e = case, _BYTES[case["dtype"]]
    if c["op"] == "rope":
        T = c["gd"] * c["gh"] * c["gw"]
        n = c["B"] * T * (c["Hq"] + c["Hk"])
        P = c["pd"] + c["ph"] + c["pw"]
        return {"bytes": 2 * n * c["D"] * e + (12 * c["B"] * T if c["positions"] else 0) + 4 * P,
                "flops": 6 * n * P}
    if c["op"] == "norm":
        n, rows = c["B"] * c["T"] * c["C"], c["B"] * c["T"]
        gate = {"batch": c["B"], "channel": 1, "none": 0}[c["gate"]] * c["C"]
        vecs = (gate + 2 * c["C"]) * e
        if c["pass"] == "forward":
            return {"bytes": 4 * n * e + vecs, "flops": 12 * n}
        # forward: x, h in, y, z out; backward: x, h, dy, dz in, dx, dh and the vectors' gradients out
        return {"bytes": 10 * n * e + 32 * rows + 2 * vecs + 4 * (gate + 2 * c["C"]),
                "flops": 36 * n}
    B, Tq, Hq, Hk, D = (c[n] for n in ("B", "Tq", "Hq", "Hk", "D"))
    kv, off, pre = _lengths(c)
    pairs = keys = 0
    for b in range(B):
        first = kv[b] - Tq
        for lo, hi, n in zip(off, off[1:], pre):
            hi = min(hi, kv[b])
            i0, i1 = max(0, lo - first), max(0, min(Tq, hi - first))
            if i0 >= i1 or lo >= hi:
                continue
            keys += hi - lo
            if not c["causal"]:
                pairs += (i1 - i0) * (hi - lo)
            else:
                pairs += sum(min(hi - lo, max(i + first + 1 - lo, n)) for i in range(i0, i1))
    qo, kvb = B * Tq * Hq * D * e, keys * Hk * D * e
    extra = 4 * B * Hq * Tq + (4 * c["axes"] * (B * Tq + keys) if c["axes"] else 0)
    if c["pass"] == "forward":
        return {"bytes": 2 * qo + 2 * kvb + extra, "flops": 4 * D * pairs * Hq}
    # forward, then q, k, v, out, dout in and dq, dk, dv out
    return {"bytes": 6 * qo + 6 * kvb + 2 * extra, "flops": 14 * D * pairs * Hq}
