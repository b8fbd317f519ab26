"""Answering from caches of a pooled volume's tokens, as cases to measure:
keys and values quantised as they are written into a cache, caches read back,
and attention of new tokens over such caches (or plain ones), behind a prefix
that several sequences share.

Each case is one pass as a serving loop makes it.  ``run`` computes it in
plain torch (elementary operations in float32, rounded once at the end), or,
where the module's ``own`` is true, by this package's kernels; ``exact``
computes it from the definition in float64.

Definitions.  Channels go in groups of 32 (the last may be shorter).  A group
x is held as 2^s and a small number for each channel, s the least integer
with max |x| <= M 2^s, not under -126:
  e4m3   1 sign, 4 exponent, 3 fraction bits, M = 448
  e2m1   1 sign, 2 exponent, 1 fraction bit, M = 6 (0 0.5 1 1.5 2 3 4 6)
each the nearest to x / 2^s (ties to the even last bit), but not past the
storage type's largest number.

  store      tokens t < count[b] go to the cache's rows start[b] + t, and are
             read back as the values that the cache then holds
  read       rows of a cache, in the storage type
  attention  query i of sequence b sees the first prefix_len[n] keys of the
             prefix n = b / (B / N), and its own keys up to
             i + kv_len[b] - Tq.  s = scale q.k, then cap tanh(s / cap), then
             minus sum_a slope[h, a] |pos_q[a, i] - pos[a, j]|; softmax over
             all keys that it sees.
"""
import math

import torch

own = False

_TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
_BYTES = {"float32": 4, "float16": 2, "bfloat16": 2}
_LARGEST = {"float32": 3.4028234663852886e38, "float16": 65504.0,
            "bfloat16": 3.3895313892515355e38}
# bits, exponent's smallest value of a normal number, fraction bits, largest number
_FORMATS = {"e4m3": (8, -6, 3, 448.0), "e2m1": (4, 0, 1, 6.0)}


def _store_case(name, dtype, fmt, B, T, Hk, D, rows, padded=False):
    return {"name": name, "op": "store", "dtype": dtype, "format": fmt, "B": B, "T": T, "Hk": Hk,
            "D": D, "rows": rows, "padded": padded}


def _read_case(name, dtype, fmt, B, T, Hk, D):
    return {"name": name, "op": "read", "dtype": dtype, "format": fmt, "B": B, "T": T, "Hk": Hk,
            "D": D}


def _attn_case(name, dtype, fmt, B, Tq, Tk, Hq, Hk, D, N=0, P=0, cap=0.0, axes=0):
    return {"name": name, "op": "attention", "dtype": dtype, "format": fmt, "B": B, "Tq": Tq,
            "Tk": Tk, "Hq": Hq, "Hk": Hk, "D": D, "N": N, "P": P, "cap": cap, "axes": axes}


def listed():
    return [
        # one new token of each of 32 sequences: latency
        _store_case("store_decode", "bfloat16", "e4m3", 32, 1, 4, 128, 1024),
        # the tokens of four (15, 27, 27) volumes, as prompts
        _store_case("store_prompt", "bfloat16", "e4m3", 4, 10935, 4, 128, 10935),
        # a padded batch of prompts, heads of 72 channels, four bits
        _store_case("store_padded_4bit", "float16", "e2m1", 5, 1330, 8, 72, 2047, padded=True),
        # a long cache for a pass that has no other use of it than plain values
        _read_case("read_long", "bfloat16", "e4m3", 2, 32768, 8, 128),
        # a short one, four bits, in float32
        _read_case("read_short_4bit", "float32", "e2m1", 2, 777, 4, 64),
        # decoding with long caches of different lengths, no shared prefix
        _attn_case("attn_long", "bfloat16", "e4m3", 16, 1, 32768, 32, 8, 128),
        # decoding at the start of one sequence: latency
        _attn_case("attn_short_4bit", "float16", "e2m1", 1, 1, 777, 16, 4, 128, cap=30.0, axes=1),
        # 32 questions about one clip of 10935 tokens, plain caches
        _attn_case("attn_clip_plain", "bfloat16", "", 32, 1, 512, 16, 4, 128, N=1, P=10935),
        # 64 continuations of one long prompt, eight bits
        _attn_case("attn_shared_wide", "bfloat16", "e4m3", 64, 1, 1024, 32, 8, 128, N=1, P=32768),
        # four clips with eight answers each, 16 drafted tokens at a time, four bits
        _attn_case("attn_draft_4bit", "bfloat16", "e2m1", 32, 16, 777, 16, 2, 128, N=4, P=6272,
                   cap=50.0),
        # questions about small pooled volumes in float32, near cells favoured on all axes
        _attn_case("attn_small_f32", "float32", "e4m3", 15, 7, 100, 12, 12, 80, N=3, P=245,
                   axes=3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("store", "read", "attention", "attention", "attention"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
    fmt = rng.choice(("e4m3", "e4m3", "e2m1"))
    D = rng.choice((32, 64, 72, 80, 96, 128, 128, 2 * rng.randint(8, 64)))
    Hk = rng.choice((1, 2, 4, 8))
    if op != "attention":
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, min(32768, 20_000_000 // (B * Hk * D))))
        if op == "read":
            return _read_case("", dtype, fmt, B, T, Hk, D)
        return _store_case("", dtype, fmt, B, T, Hk, D, T + rng.randint(0, 1000),
                           padded=rng.random() < 0.5)
    Hq = Hk * rng.choice((1, 2, 4, 8)) if Hk < 8 else rng.choice((8, 16, 32))
    fmt = rng.choice((fmt, fmt, ""))
    N = rng.choice((0, 1, 1, rng.randint(1, 6)))
    B = _log_int(rng, 1, 64)
    if N:
        B = max(1, B // N) * N
    Tq = rng.choice((1, 1, 1, rng.randint(2, 32)))
    # pairs of a query and a key, and elements of the caches, bounded
    most = max(Tq, min(32768, 60_000_000 // (B * Tq * Hq), 1_000_000 // (Hk * max(N, 1))))
    P = _log_int(rng, min(16, most), most) if N else 0
    most = max(Tq, min(32768, 30_000_000 // (B * Tq * Hq), 60_000_000 // (Hk * D * B)))
    Tk = max(Tq, _log_int(rng, min(16, most), most))
    return _attn_case("", dtype, fmt, B, Tq, Tk, Hq, Hk, D, N=N, P=P,
                      cap=rng.choice((0.0, 0.0, 30.0)), axes=rng.choice((0, 0, 0, 1, 3)))


# ---------------------------------------------------------------- inputs

def _counts(case):
    """Host lists that a case implies: tokens in use of each sequence, and of
    each prefix."""
    B = case["B"]
    if case["op"] == "store":
        n = case["T"]
        return [n - (b * (n // 2)) // B if case["padded"] else n for b in range(B)], []
    if case["op"] == "read":
        return [case["T"]] * B, []
    least, most = case["Tq"], case["Tk"]
    kv = [max(least, most - (b * (3 * most // 4)) // B) for b in range(B)]
    pre = [case["P"] - (n * (case["P"] // 4)) // case["N"] for n in range(case["N"])]
    return kv, pre


def _rand(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _keys(shape, gen, dtype):
    """Keys with a few channels of each head larger than the rest."""
    big = torch.rand((1, 1) + shape[2:], generator=gen, device="cuda") < 0.05
    return (torch.randn(shape, generator=gen, device="cuda") * (1.0 + 3.0 * big)).to(dtype)


def _power(e):
    """2^e in float32, for integers -126 <= e <= 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _numbers(fmt, device):
    """The values of all codes, in float32."""
    bits, low, frac, _ = _FORMATS[fmt]
    code = torch.arange(1 << bits, device=device)
    f = (code & ((1 << frac) - 1)).float() / (1 << frac)
    e = (code >> frac) & ((1 << (bits - 1 - frac)) - 1)
    size = torch.where(e == 0, f * 2.0 ** low, (1.0 + f) * _power(e - 1 + low))
    if fmt == "e4m3":
        size = size.masked_fill((code & 127) == 127, float("nan"))
    return torch.where(code >> (bits - 1) == 1, -size, size)


def _split(x, fmt, dtype):
    """Groups of 32 channels of x (float32): the exponents s (int32), and
    x / 2^s rounded to the format's numbers."""
    _, low, frac, top = _FORMATS[fmt]
    D = x.shape[-1]
    g = torch.nn.functional.pad(x, (0, -D % 32)).unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1)
    m, e = torch.frexp(amax)
    mt, et = math.frexp(top)
    s = (e - et + (m > mt).to(torch.int32)).clamp(min=-126)
    y = g * _power(-s)[..., None]
    _, e = torch.frexp(y.abs())
    step = (e - 1).clamp(min=low) - frac
    q = torch.round(y * _power(-step)) * _power(step)
    # (2^s times the format's largest number but one binade may be past the type)
    over = 2.0 ** math.floor(math.log2(top))                  # 256 or 4
    last = over * (2.0 - 2.0 ** -frac) / 2.0                  # 240 or 3
    past = (over * torch.exp2(s.double()) > _LARGEST[dtype])[..., None]
    q = torch.where(past, q.clamp(-last, last), q.clamp(-top, top))
    return s, q


def _plain_values(x, fmt, dtype):
    s, q = _split(x.float(), fmt, dtype)
    return (q * _power(s)[..., None]).flatten(-2)[..., :x.shape[-1]].to(x.dtype)


def _encode(x, fmt, dtype):
    """x (B, T, H, D) as codes and scales, laid out head by head: (B, T, H, .)
    views of (B, H, T, .)."""
    B, T, H, D = x.shape
    width = D if fmt == "e4m3" else (D + 1) // 2
    codes = torch.empty((B, H, T, width), dtype=torch.uint8, device=x.device).transpose(1, 2)
    scales = torch.empty((B, H, T, -(-D // 32)), dtype=torch.uint8,
                         device=x.device).transpose(1, 2)
    for b in range(B):
        s, q = _split(x[b].float(), fmt, dtype)
        scales[b] = (s + 127).to(torch.uint8)
        q = q.flatten(-2)
        if fmt == "e4m3":
            codes[b] = q[..., :D].to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
            c = torch.bucketize(q.abs(), steps) + 8 * (q < 0)
            codes[b] = (c[..., 0::2] + 16 * c[..., 1::2])[..., :width].to(torch.uint8)
    return codes, scales


def _cache(B, T, Hk, D, fmt, dtype, gen):
    """What a program keeps of B sequences: (k, v), or codes and scales of
    both."""
    dt = _TYPES[dtype]
    if not fmt:
        return (_keys((B, Hk, T, D), gen, dt).transpose(1, 2),
                _rand((B, Hk, T, D), gen, dt).transpose(1, 2))
    parts = []
    for make in (_keys, _rand):
        per = max(1, 40_000_000 // max(1, T * Hk * D))
        some = [_encode(make((min(per, B - b), T, Hk, D), gen, dt), fmt, dtype)
                for b in range(0, B, per)]
        for i in range(2):
            parts.append(some[0][i] if len(some) == 1
                         else torch.cat([x[i].transpose(1, 2) for x in some]).transpose(1, 2))
    return tuple(parts)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]
    dev = "cuda"
    B, Hk, D = case["B"], case["Hk"], case["D"]
    st = {"case": case}
    used, pre = _counts(case)
    if case["op"] == "store":
        T = case["T"]
        # k and v as the two ends of one projection's output
        kv = _rand((B, T, 2 * Hk, D), gen, dt)
        kv[:, :, :Hk] = _keys((B, T, Hk, D), gen, dt)
        st["k"], st["v"] = kv[:, :, :Hk], kv[:, :, Hk:]
        st["cache"] = _cache(B, case["rows"], Hk, D, case["format"], case["dtype"], gen)
        st["start"] = torch.randint(0, case["rows"] - T + 1, (B,), generator=gen, device=dev,
                                    dtype=torch.int32)
        st["count"] = (torch.tensor(used, dtype=torch.int32, device=dev) if case["padded"]
                       else None)
        return st
    if case["op"] == "read":
        st["cache"] = _cache(B, case["T"], Hk, D, case["format"], case["dtype"], gen)
        return st
    Hq, Tq, Tk, N, P, A = (case[n] for n in ("Hq", "Tq", "Tk", "N", "P", "axes"))
    st["q"] = _rand((B, Tq, Hq, D), gen, dt)
    st["own"] = _cache(B, Tk, Hk, D, case["format"], case["dtype"], gen)
    st["prefix"] = _cache(N, P, Hk, D, case["format"], case["dtype"], gen) if N else None
    st["kv_len"] = torch.tensor(used, dtype=torch.int32, device=dev)
    st["prefix_len"] = torch.tensor(pre, dtype=torch.int32, device=dev) if N > 1 else None
    st["pos_q"] = st["pos_k"] = st["pos_prefix"] = st["slopes"] = None
    if A:
        # the prefix' cells in a volume 27 cells high and wide, own tokens after them
        t = torch.arange(P + Tk, device=dev, dtype=torch.int32)
        cell = torch.stack((t // 729, t // 27 % 27, t % 27)) if A == 3 else t[None]
        at = st["kv_len"].long()[:, None] - Tq + torch.arange(Tq, device=dev)
        st["pos_q"] = cell[:, P:][:, at].contiguous()
        st["pos_k"] = cell[:, None, P:].expand(A, B, Tk).contiguous()
        if N:
            st["pos_prefix"] = cell[:, None, :P].expand(A, N, P).contiguous()
        st["slopes"] = (torch.rand((Hq, A), generator=gen, device=dev) + 0.5) * (
            2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq))[:, None]
    return st


# ----------------------------------------------------------------- passes

def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["op"]](state, case)


def _own_store(st, c):
    import bwd_max_pool3d_amd as mp
    mp.mp3d_cache_write(st["k"], st["v"], st["cache"], c["format"], start=st["start"],
                        count=st["count"])
    return mp.mp3d_cache_read(st["cache"], c["format"], c["D"], st["k"].dtype, rows=c["T"],
                              start=st["start"], count=st["count"])


def _own_read(st, c):
    import bwd_max_pool3d_amd as mp
    return mp.mp3d_cache_read(st["cache"], c["format"], c["D"], _TYPES[c["dtype"]])


def _own_attention(st, c):
    import bwd_max_pool3d_amd as mp
    return mp.mp3d_attention_cached(st["q"], st["own"], st["prefix"], format=c["format"] or None,
                                    softcap=c["cap"], kv_len=st["kv_len"],
                                    prefix_len=st["prefix_len"], slopes=st["slopes"],
                                    pos_q=st["pos_q"], pos_k=st["pos_k"],
                                    pos_prefix=st["pos_prefix"])


_own = {"store": _own_store, "read": _own_read, "attention": _own_attention}


def _plain_store(st, c):
    outs = []
    for n in ("k", "v"):
        x = _plain_values(st[n], c["format"], c["dtype"])
        if st["count"] is not None:
            t = torch.arange(c["T"], device=x.device)
            x = torch.where((t < st["count"][:, None])[..., None, None], x, torch.zeros_like(x))
        outs.append(x)
    return tuple(outs)


def _decode(codes, scales, fmt, D):
    """float32 values of codes and scales."""
    table = _numbers(fmt, codes.device)
    if fmt == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)[..., :D]
    x = table[codes.int()]
    scale = _power(scales.int() - 127).repeat_interleave(32, -1)[..., :D]
    return x * scale


def _plain_read(st, c):
    kc, ks, vc, vs = st["cache"]
    dt = _TYPES[c["dtype"]]
    return tuple(_decode(a, b, c["format"], c["D"]).to(dt).contiguous()
                 for a, b in ((kc, ks), (vc, vs)))


def _floats(cache, fmt, D):
    """Keys and values (B, H, T, D) of a cache in float32."""
    if fmt:
        cache = _decode(cache[0], cache[1], fmt, D), _decode(cache[2], cache[3], fmt, D)
    return tuple(x.float().transpose(1, 2).contiguous() for x in cache)


def _plain_attention(st, c):
    q = st["q"]
    B, Tq, Hq, D = q.shape
    Hk, Tk, N, P = c["Hk"], c["Tk"], c["N"], c["P"]
    G, scale = Hq // Hk, 1.0 / math.sqrt(D)
    qf = (q.float() * scale).view(B, Tq, Hk, G, D).permute(0, 2, 1, 3, 4).contiguous()

    def scores(x, k, pos_q, pos_k, hide):
        """(n, Hk, rows..., Tq, G, keys) scores of x against k, masked."""
        shape = x.shape[:-1] + (k.shape[2],)
        s = (x.flatten(2, -2) @ k.transpose(2, 3).contiguous()).view(shape)
        if c["cap"]:
            s = c["cap"] * torch.tanh(s / c["cap"])
        if st["slopes"] is not None:
            far = (pos_q[..., :, None] - pos_k[..., None, :]).abs().float()
            bias = st["slopes"] @ far.view(far.shape[0], -1)
            bias = bias.view((Hk, G) + far.shape[1:])
            # (Hk, G, n, rows..., Tq, keys) -> (n, Hk, rows..., Tq, G, keys)
            s = s - bias.movedim(1, -2).movedim(0, 1)
        return s.masked_fill(hide, float("-inf"))

    kv_len = st["kv_len"].long()
    k, v = _floats(st["own"], c["format"], D)
    j = torch.arange(Tk, device=q.device)
    last = kv_len[:, None] - Tq + torch.arange(Tq, device=q.device)
    hide = (j > last[..., None])[:, None, :, None]
    s = scores(qf, k, st["pos_q"], st["pos_k"], hide).flatten(2, 3)      # (B, Hk, Tq G, Tk)
    if N:
        S = B // N
        kp, vp = _floats(st["prefix"], c["format"], D)
        rows = qf.view(N, S, Hk, Tq, G, D).transpose(1, 2).contiguous()
        length = (torch.full((N,), P, device=q.device) if st["prefix_len"] is None
                  else st["prefix_len"].long())
        hide = (torch.arange(P, device=q.device) >= length[:, None])[:, None, None, None, None]
        A = c["axes"]
        sp = scores(rows, kp, st["pos_q"].view(A, N, S, Tq) if A else None,
                    st["pos_prefix"][:, :, None] if A else None, hide)
        sp = sp.transpose(1, 2).reshape(B, Hk, Tq * G, P)
        s = torch.cat((sp, s), -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).view(B, Hk, Tq, G).transpose(2, 3).reshape(B, Hq, Tq)
    p = p / total
    o = p[..., P:] @ v
    if N:
        w = p[..., :P].reshape(N, S, Hk, Tq * G, P).transpose(1, 2).reshape(N, Hk, -1, P)
        o = o + (w @ vp).view(N, Hk, S, Tq * G, D).transpose(1, 2).reshape(B, Hk, Tq * G, D)
    out = o.view(B, Hk, Tq, G, D).transpose(1, 2).reshape(B, Tq, Hq, D).to(q.dtype).contiguous()
    return out, lse


_plain = {"store": _plain_store, "read": _plain_read, "attention": _plain_attention}


# -------------------------------------------------------------- definitions

def exact(case, seed):
    st = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "attention": _exact_attention}[case["op"]](
        st, case)


def _magnitudes(fmt):
    """The format's numbers >= 0 in the order of their codes."""
    if fmt == "e2m1":
        return [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    sub = [i * 2.0 ** -9 for i in range(8)]
    return sub + [(8 + i) * 2.0 ** (e - 10) for e in range(1, 16) for i in range(8)][:-1]


def _exact_store(st, c):
    mags = torch.tensor(_magnitudes(c["format"]), dtype=torch.float64, device=st["k"].device)
    middle = (mags[1:] + mags[:-1]) / 2
    top, largest = float(mags[-1]), _LARGEST[c["dtype"]]
    used, _ = _counts(c)
    outs = []
    for n in ("k", "v"):
        x = st[n]
        y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        for b in range(c["B"]):
            for lo in range(0, c["D"], 32):
                g = x[b, :used[b], :, lo:lo + 32].double()
                a = g.abs().amax(-1, keepdim=True)
                s = torch.ceil(torch.log2((a / top).clamp(min=2.0 ** -130)))
                s = torch.where(torch.exp2(s - 1) * top >= a, s - 1, s)
                s = torch.where(torch.exp2(s) * top < a, s + 1, s).clamp(min=-126)
                unit = torch.exp2(s)
                r = g.abs() / unit
                i = torch.searchsorted(middle, r.contiguous())           # middle[i - 1] < r <= middle[i]
                tie = r == middle[i.clamp(max=len(middle) - 1)]
                i = torch.where(tie & (i % 2 == 1), i + 1, i)
                z = mags[i] * unit
                # numbers past the type's largest: the one of the format below them
                below = torch.where(unit * mags <= largest, mags, 0.0).amax(
                    -1, keepdim=True) * unit
                y[b, :used[b], :, lo:lo + 32] = torch.sign(g) * torch.minimum(z, below)
        outs.append(y)
    return tuple(outs)


def _exact_values(codes, scales, fmt, D):
    """float64 values (T, D) of one head."""
    half = torch.tensor(_magnitudes(fmt) + ([float("nan")] if fmt == "e4m3" else []),
                        dtype=torch.float64, device=codes.device)
    table = torch.cat((half, -half))
    c = codes.long()
    if fmt == "e2m1":
        both = torch.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=torch.long, device=c.device)
        both[..., 0::2], both[..., 1::2] = c % 16, c // 16
        c = both[..., :D]
    unit = torch.exp2(scales.double() - 127.0)
    return table[c] * unit[..., torch.arange(D, device=c.device) // 32]


def _exact_read(st, c):
    kc, ks, vc, vs = st["cache"]
    outs = []
    for a, b in ((kc, ks), (vc, vs)):
        y = torch.empty(c["B"], c["T"], c["Hk"], c["D"], dtype=torch.float64, device=a.device)
        for i in range(c["B"]):
            for h in range(c["Hk"]):
                y[i, :, h] = _exact_values(a[i, :, h], b[i, :, h], c["format"], c["D"])
        outs.append(y)
    return tuple(outs)


def _exact_attention(st, c):
    q = st["q"]
    B, Tq, Hq, D = q.shape
    Hk, N = c["Hk"], c["N"]
    used, pre = _counts(c)
    dev, f64 = q.device, torch.float64
    out = torch.zeros(B, Tq, Hq, D, dtype=f64, device=dev)
    lse = torch.zeros(B, Hq, Tq, dtype=f64, device=dev)

    def head(cache, i, g, length):
        if c["format"]:
            return tuple(_exact_values(cache[2 * x][i, :length, g], cache[2 * x + 1][i, :length, g],
                                       c["format"], D) for x in range(2))
        return cache[0][i, :length, g].double(), cache[1][i, :length, g].double()

    for g in range(Hk):
        for b in range(B):
            if N and b % (B // N) == 0:
                n = b // (B // N)
                kp, vp = head(st["prefix"], n, g, pre[n])
            k, v = head(st["own"], b, g, used[b])
            P = 0
            if N:
                k, v, P = torch.cat((kp, k)), torch.cat((vp, v)), pre[n]
            j = torch.arange(used[b], device=dev)
            i = torch.arange(Tq, device=dev) + used[b] - Tq
            hide = torch.cat((torch.zeros(Tq, P, dtype=torch.bool, device=dev),
                              j[None] > i[:, None]), 1)
            heads = range(g * (Hq // Hk), (g + 1) * (Hq // Hk))
            x = torch.cat([q[b, :, h].double() for h in heads])
            s = torch.matmul(x, k.t()) / math.sqrt(D)
            if c["cap"]:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if st["slopes"] is not None:
                for a in range(c["axes"]):
                    pk = st["pos_k"][a, b, :used[b]].double()
                    if N:
                        pk = torch.cat((st["pos_prefix"][a, n, :P].double(), pk))
                    gap = (st["pos_q"][a, b].double()[:, None] - pk[None]).abs()
                    s = s - torch.cat([float(st["slopes"][h, a].double()) * gap for h in heads])
            s = torch.where(hide.repeat(len(heads), 1), torch.full_like(s, float("-inf")), s)
            o = torch.matmul(torch.softmax(s, 1), v).view(len(heads), Tq, D)
            out[b, :, heads[0]:heads[-1] + 1] = o.transpose(0, 1)
            lse[b, heads[0]:heads[-1] + 1] = torch.logsumexp(s, 1).view(len(heads), Tq)
    return out, lse


# --------------------------------------------------------------------- work

def work(case):
    c, e = case, _BYTES[case["dtype"]]
    D, Hk = c["D"], c["Hk"]
    # bytes of a token's key (or value) in the cache
    if c["format"]:
        held = Hk * ((D if c["format"] == "e4m3" else (D + 1) // 2) + -(-D // 32))
    else:
        held = Hk * D * e
    used, pre = _counts(c)
    if c["op"] == "store":
        n = sum(used)
        # k and v in, the cache's rows and their values out
        return {"bytes": 2 * n * (Hk * D * e + held) + 2 * c["B"] * c["T"] * Hk * D * e,
                "flops": 4 * 2 * n * Hk * D}
    if c["op"] == "read":
        n = c["B"] * c["T"]
        return {"bytes": 2 * n * (held + Hk * D * e), "flops": 2 * n * Hk * D}
    B, Tq, Hq, N = c["B"], c["Tq"], c["Hq"], c["N"]
    pairs = 0
    for b in range(B):
        pairs += Tq * used[b] - Tq * (Tq - 1) // 2 + (Tq * pre[b // (B // N)] if N else 0)
    keys = sum(used) + sum(pre)
    return {"bytes": 2 * keys * held + 2 * B * Tq * Hq * D * e + 4 * B * Tq * Hq
            + 4 * c["axes"] * (B * Tq + keys), "flops": 4 * D * pairs * Hq}
