"""Attention and its backward against the float64 form: types, head layouts,
lengths around every tile's edge, masks that leave rows empty, caches,
infinities and NaN in masked places."""
import pytest
import torch

import _tokens as tk
import bwd_max_pool3d_amd as mp

pytestmark = pytest.mark.gpu


def make(B, Tq, Tk, Hq, Hk, D, dt, seed):
    return (tk.randn((B, Tq, Hq, D), seed, dt), tk.randn((B, Tk, Hk, D), seed + 1, dt),
            tk.randn((B, Tk, Hk, D), seed + 2, dt), tk.randn((B, Tq, Hq, D), seed + 3, dt))


def dev(how):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in how.items()}


def run(q, k, v, do, how):
    d = dev(how)
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    out, lse = mp.mp3d_attention_forward(q, k, v, **d)
    dq, dk, dv = mp.mp3d_attention_backward(do, q, k, v, out, lse, **d)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def check(q, k, v, do, how):
    got = run(q, k, v, do, how)
    for name, (value, tol) in tk.attention(q, k, v, do, **how).items():
        tk.close(got[name], value, tol, name)


def bias(B, Tq, Tk, Hq, axes, seed):
    g = torch.Generator().manual_seed(seed)
    j = torch.arange(Tk)
    cells = torch.stack((j // 30, j // 6 % 5, j % 6))[:axes] if axes > 1 else j[None]
    pk = cells[:, None].expand(axes, B, Tk).contiguous().int()
    pq = torch.randint(0, max(Tk, 1), (axes, B, Tq), generator=g, dtype=torch.int32)
    return dict(slopes=torch.rand((Hq, axes), generator=g) * 0.2, pos_q=pq, pos_k=pk)


# (B, Tq, Tk, Hq, Hk, D)
SHAPES = [
    (1, 1, 1, 1, 1, 1), (2, 1, 37, 4, 2, 64), (1, 3, 64, 2, 1, 8), (1, 31, 31, 2, 2, 40),
    (1, 33, 65, 3, 1, 65), (2, 64, 64, 2, 2, 128), (1, 127, 129, 2, 1, 80),
    (1, 129, 127, 2, 2, 127), (1, 200, 300, 4, 1, 64), (1, 300, 200, 1, 1, 96),
    (3, 5, 1100, 6, 2, 128), (1, 70, 1500, 2, 1, 72), (1, 257, 513, 2, 2, 64),
]


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_shapes(shape, dt, causal):
    check(*make(*shape, dt, 40), dict(causal=causal))


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("shape", [(2, 1, 300, 8, 2, 64), (1, 150, 150, 2, 1, 64),
                                   (1, 100, 260, 2, 2, 128)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("what", ["cap", "bias1", "bias2", "bias3", "cap+bias3", "scale",
                                  "negative", "zero"])
def test_scores(shape, dt, what):
    B, Tq, Tk, Hq, Hk, D = shape
    how = dict(causal=True)
    if "cap" in what:
        how.update(softcap=1.5)
    for n in (1, 2, 3):
        if "bias%d" % n in what:
            how.update(bias(B, Tq, Tk, Hq, n, 41))
    if what == "scale":
        how.update(scale=0.7)
    if what == "negative":
        how.update(scale=-0.3)
    if what == "zero":
        how.update(scale=0.0)
    check(*make(*shape, dt, 42), how)


DOCS = [
    [[0, 200]], [[0, 1, 2, 64, 64, 128, 200]], [[10, 50, 50, 190]], [[0, 33, 97, 161, 199]],
    [[0, 0, 0, 200]], [[200, 200]], [[0, 0]], [[-5, 60, 900]],
]


@pytest.mark.parametrize("causal,prefix", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("docs", DOCS, ids=str)
def test_documents(docs, causal, prefix):
    how = dict(causal=causal, doc_offsets=torch.tensor(docs, dtype=torch.int32))
    if prefix:
        g = torch.Generator().manual_seed(43)
        how["prefix"] = torch.randint(0, 50, (1, len(docs[0]) - 1), generator=g, dtype=torch.int32)
    for dt in (torch.float32, torch.bfloat16):
        check(*make(1, 200, 200, 2, 1, 64, dt, 44), how)


def test_documents_differ_by_sequence():
    docs = torch.tensor([[0, 30, 100], [0, 90, 95], [40, 40, 41]], dtype=torch.int32)
    check(*make(3, 100, 100, 2, 2, 64, torch.float16, 45),
          dict(causal=True, doc_offsets=docs, **bias(3, 100, 100, 2, 3, 46)))


@pytest.mark.parametrize("prefix", [[0, 0], [1, 64], [65, 150], [1000000000, -3]], ids=str)
@pytest.mark.parametrize("Tq", [1, 150])
def test_prefix(prefix, Tq):
    how = dict(causal=True, prefix=torch.tensor(prefix, dtype=torch.int32))
    check(*make(2, Tq, 150, 4, 2, 64, torch.bfloat16, 47), how)


@pytest.mark.parametrize("Tq", [1, 2, 9, 70, 300])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=tk.name_of)
@pytest.mark.parametrize("causal", [False, True])
def test_kv_len(Tq, dt, causal):
    """Caches in part in use: none, one, less than the queries, all, more
    than there is; the rest of the cache holds NaN and is not read."""
    lens = [0, 1, 5, 257, 300, 1000]
    q, k, v, do = make(6, Tq, 300, 4, 1, 64, dt, 48)
    how = dict(causal=causal, kv_len=torch.tensor(lens, dtype=torch.int32))
    clean = tk.attention(q, k, v, do, **how)
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = float("nan"), float("inf")
    got = run(q, k, v, do, how)
    for name, (value, tol) in clean.items():
        tk.close(got[name], value, tol, name)
    assert torch.equal(got["out"][0].cpu(), torch.zeros_like(q[0]))
    assert bool((got["lse"][0] == float("-inf")).all())
    assert torch.equal(got["dk"][1, 1:].cpu(), torch.zeros_like(k[1, 1:]))


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("Tq", [2, 180])
def test_nonfinite_in_masked_places(value, dt, Tq):
    """A key or value that is not finite changes nothing for the queries that
    do not see it, in the forward and in dq; a gradient that is not finite
    changes nothing for the keys its query does not see."""
    Tk, at = 180, 178 if Tq == 2 else 100
    q, k, v, do = make(1, Tq, Tk, 4, 2, 64, dt, 49)
    how = dict(causal=True)
    clean = run(q, k, v, do, how)
    k2, v2 = k.clone(), v.clone()
    v2[0, at + 1, :, 3] = value
    got = run(q, k, v2, do, how)
    see = at + 1 - (Tk - Tq)                             # the first query that sees that key
    assert torch.equal(got["out"][:, :see], clean["out"][:, :see])
    assert not torch.isfinite(got["out"][:, see:, :, 3]).any()
    others = [d for d in range(64) if d != 3]
    assert torch.equal(got["out"][..., others], clean["out"][..., others])
    assert torch.equal(got["dq"][:, :see], clean["dq"][:, :see])
    assert not torch.isfinite(got["dq"][:, see:]).any()
    k2[0, at + 1, :, 5] = value
    got = run(q, k2, v, do, how)
    assert torch.equal(got["out"][:, :see], clean["out"][:, :see])
    assert torch.equal(got["dq"][:, :see], clean["dq"][:, :see])
    # the gradient of the last-but-one query: keys after it
    do2 = do.clone()
    do2[0, Tq - 2, :, 7] = value
    got = run(q, k, v, do2, how)
    last = Tk - 1
    assert torch.equal(got["dv"][:, last:], clean["dv"][:, last:])
    assert torch.equal(got["dk"][:, last:], clean["dk"][:, last:])
    assert not torch.isfinite(got["dv"][:, :last, :, 7]).any()
    assert not torch.isfinite(got["dk"][:, :last]).any()
    assert torch.equal(got["dq"][:, Tq - 1:], clean["dq"][:, Tq - 1:])


def test_scores_of_minus_infinity():
    """A query whose every visible score is -infinity gives 0 and -infinity,
    and no gradient."""
    q, k, v, do = make(1, 80, 80, 1, 1, 64, torch.float32, 50)
    k[..., 0] = -float("inf")
    q[..., 0] = q[..., 0].abs() + 0.1
    got = run(q, k, v, do, dict(causal=True))
    assert torch.equal(got["out"].cpu(), torch.zeros_like(q))
    assert bool((got["lse"] == float("-inf")).all())
    assert torch.equal(got["dv"].cpu(), torch.zeros_like(v))


@pytest.mark.parametrize("layout", ["head_major", "qkv", "misaligned", "expanded"])
@pytest.mark.parametrize("Tq", [1, 90])
def test_layouts(layout, Tq):
    B, Tk, H, D, dt = 2, 90, 4, 64, torch.bfloat16
    q, k, v, do = make(B, Tq, Tk, H, H, D, dt, 51)
    how = dict(causal=True)
    if layout == "head_major":
        ten = [t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (q, k, v, do)]
    elif layout == "misaligned":
        ten = [torch.nn.functional.pad(t, (1, 4)).cuda()[..., 1:1 + D] for t in (q, k, v, do)]
    elif layout == "expanded":                       # one head's gradient for all, one key head
        k, v, do = (t[:, :, :1].expand(-1, -1, H, -1) for t in (k, v, do))
        ten = [q.cuda()] + [t[:, :, :1].contiguous().cuda().expand(-1, -1, H, -1)
                            for t in (k, v, do)]
    else:
        kv = torch.cat((k, v), 2).cuda()
        ten = [q.cuda(), kv[:, :, :H], kv[:, :, H:], do.cuda()]
    out, lse = mp.mp3d_attention_forward(*ten[:3], **how)
    g = mp.mp3d_attention_backward(ten[3], *ten[:3], out, lse, **how)
    got = dict(zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + g))
    for name, (value, tol) in tk.attention(q, k, v, do, **how).items():
        tk.close(got[name], value, tol, name)


@pytest.mark.parametrize("shape", [(1, 1, 4000, 8, 1, 128), (2, 4, 2100, 16, 2, 64),
                                   (1, 40, 3000, 8, 8, 96), (1, 1, 8000, 32, 32, 64)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
def test_split(shape, dt):
    """Few queries over many keys: split over the keys and joined."""
    B, Tq, Tk, Hq, Hk, D = shape
    q, k, v, do = make(*shape, dt, 52)
    how = dict(causal=True, softcap=20.0, kv_len=torch.tensor([Tk - 37 * b for b in range(B)],
                                                              dtype=torch.int32))
    how.update(bias(B, Tq, Tk, Hq, 1, 53))
    out, lse = mp.mp3d_attention_forward(q.cuda(), k.cuda(), v.cuda(), **dev(how))
    want = tk.attention(q, k, v, **how)
    tk.close(out, *want["out"], "out")
    tk.close(lse, *want["lse"], "lse")


def test_growing_scores():
    """Scores that rise along the keys by far more than the running maximum's
    slack, and fall again."""
    for dt in tk.TYPES:
        q, k, v, do = make(1, 100, 300, 1, 1, 32, dt, 54)
        ramp = torch.linspace(0, 40, 300)[None, :, None, None]
        q = q.abs() + 0.5
        check(q.to(dt), (k * 0.1 + ramp * 0.1).to(dt), v, do, {})
        check(q.to(dt), (k * 0.1 - ramp * 0.1).to(dt), v, do, {})


def test_repeats_bit_for_bit():
    q, k, v, do = make(2, 200, 200, 8, 2, 128, torch.bfloat16, 55)
    how = dict(causal=True)
    a, b = run(q, k, v, do, how), run(q, k, v, do, how)
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_another_stream_and_workspace():
    """Work goes to the current stream; a lent workspace may hold anything."""
    q, k, v, do = (t.cuda() for t in make(1, 4, 3000, 8, 2, 64, torch.float16, 56))
    ref = mp.mp3d_attention_forward(q, k, v, causal=True)
    n = mp.mp3d_attention_workspace_bytes(q, k, v, causal=True)
    assert n > 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mp.mp3d_attention_forward(q, k, v, causal=True, workspace=ws)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    nb = mp.mp3d_attention_workspace_bytes(q, k, v, True, causal=True)
    g0 = mp.mp3d_attention_backward(do, q, k, v, *ref, causal=True)
    g1 = mp.mp3d_attention_backward(do, q, k, v, *ref, causal=True, workspace=torch.full(
        (nb,), 255, dtype=torch.uint8, device="cuda"))
    for x, y in zip(g0, g1):
        assert torch.equal(x, y)


def test_empty():
    for B, Tq, Tk in ((0, 3, 3), (2, 0, 3), (2, 3, 0)):
        q, k, v, do = (t.cuda() for t in make(B, Tq, Tk, 2, 2, 8, torch.float32, 57))
        out, lse = mp.mp3d_attention_forward(q, k, v)
        assert torch.equal(out, torch.zeros_like(q)) and bool((lse == float("-inf")).all())
        dq, dk, dv = mp.mp3d_attention_backward(do, q, k, v, out, lse)
        assert torch.equal(dq, torch.zeros_like(q)) and torch.equal(dk, torch.zeros_like(k))
        assert torch.equal(dv, torch.zeros_like(v))


def test_gradient_against_differences():
    """<gradient, direction> against a central difference of the forward, with
    cap and bias.  The step is 2^-6: its square, 2.4e-4, times third
    derivatives of order one, and float32's error over the step, about 1e-5,
    of the size of |gradient| |direction|."""
    shape = (1, 24, 24, 2, 1, 16)
    q, k, v, do = make(*shape, torch.float32, 58)
    how = dict(causal=True, softcap=3.0, **bias(1, 24, 24, 2, 3, 59))
    got = run(q, k, v, do, how)

    def loss(q, k, v):
        out, _ = mp.mp3d_attention_forward(q.cuda(), k.cuda(), v.cuda(), **dev(how))
        return (out.double().cpu() * do.double()).sum()

    t = {"q": q, "k": k, "v": v}
    for name in t:
        d = tk.randn(t[name].shape, 60, torch.float32)
        up, down = dict(t), dict(t)
        up[name], down[name] = t[name] + d / 64, t[name] - d / 64
        diff = (loss(**up) - loss(**down)) * 32
        step = (up[name].double() - down[name].double()) * 32
        grad = got["d" + name].cpu().double()
        assert abs(diff - (grad * step).sum()) <= 1e-3 * grad.norm() * step.norm(), name
