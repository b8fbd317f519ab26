"""The token operators at the ends of their ranges: no queries, no rows, more
rows than one launch takes, keys that are not finite."""
import ctypes

import pytest
import torch

import _tokens as tk
import bwd_max_pool3d_amd as mp
from bwd_max_pool3d_amd import _lib
from test_gpu_attention import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Tk", [1, 128, 129, 700])
def test_backward_without_queries_in_documents(Tk):
    """No query: dk and dv are zeros in every block of keys, also with a
    workspace that is larger than needed and holds other numbers."""
    q, k, v, do = (t.cuda() for t in make(2, 0, Tk, 2, 2, 64, torch.float32, 75))
    docs = torch.tensor([[0, Tk // 2, Tk]] * 2, dtype=torch.int32, device="cuda")
    out, lse = mp.mp3d_attention_forward(q, k, v, doc_offsets=docs)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    grads = [torch.full(t.shape, float("nan"), device="cuda") for t in (q, k, v)]
    mp.mp3d_attention_backward(do, q, k, v, out, lse, doc_offsets=docs, grads=grads, workspace=ws)
    assert torch.equal(grads[1], torch.zeros_like(k)) and torch.equal(grads[2], torch.zeros_like(v))


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("Hq,Hk", [(4, 4), (8, 2)])
@pytest.mark.parametrize("Tk", [3, 300])
@pytest.mark.parametrize("more", ["", "documents", "bias"])
def test_backward_without_queries(more, Tk, Hq, Hk, dt):
    """No query, the workspace that the call itself asks for: shared heads,
    documents and a bias take some."""
    q, k, v, do = (t.cuda() for t in make(2, 0, Tk, Hq, Hk, 64, dt, 76))
    how = {}
    if more == "documents":
        how["doc_offsets"] = torch.tensor([[0, Tk]] * 2, dtype=torch.int32, device="cuda")
    if more == "bias":
        how["slopes"] = torch.ones((Hq, 2), device="cuda")
        how["pos_q"] = torch.zeros((2, 2, 0), dtype=torch.int32, device="cuda")
        how["pos_k"] = torch.ones((2, 2, Tk), dtype=torch.int32, device="cuda")
    out, lse = mp.mp3d_attention_forward(q, k, v, **how)
    dq, dk, dv = mp.mp3d_attention_backward(do, q, k, v, out, lse, **how)
    assert dq.shape == q.shape
    assert torch.equal(dk, torch.zeros_like(k)) and torch.equal(dv, torch.zeros_like(v))


def test_backward_of_more_rows_than_one_launch_takes():
    """553 million rows of queries: the rows' constants take 2^32 threads and
    more.  Sequences from both sides of every 2^23 workgroups, and the last,
    give the bits of a call by themselves."""
    B, Tq, H = 540000, 128, 8
    assert Tq // 32 * B * H * 256 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(77)
    q, do = (torch.randn((B, Tq, H, 1), dtype=torch.float16, device="cuda", generator=g)
             for _ in range(2))
    k, v = (torch.randn((B, 2, H, 1), dtype=torch.float16, device="cuda", generator=g)
            for _ in range(2))
    out, lse = mp.mp3d_attention_forward(q, k, v)
    grads = mp.mp3d_attention_backward(do, q, k, v, out, lse)
    per = Tq // 32 * H                                     # workgroups of a sequence
    for b in (0, (1 << 23) // per, (1 << 23) // per - 1, (1 << 24) // per, B - 1):
        one = [t[b:b + 1].contiguous() for t in (do, q, k, v, out, lse)]
        o1 = mp.mp3d_attention_forward(*one[1:4])
        assert torch.equal(o1[0], one[4]) and torch.equal(o1[1], one[5])
        for whole, part in zip(grads, mp.mp3d_attention_backward(*one)):
            assert torch.equal(whole[b:b + 1], part)
            assert part.abs().sum() > 0


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("D", [64, 128])
def test_dq_of_a_key_with_score_minus_infinity(D, dt):
    """A key whose score is -infinity has no weight: the gradient of every
    query that sees it, in all other channels, is as if the key were not
    there.  Its tile is seen in part by some waves of the first workgroup, in
    full by others, and in full by the whole second workgroup."""
    T, at = 200, 70
    q, k, v, do = make(1, T, T, 1, 1, D, dt, 66)
    q[..., 0] = q[..., 0].abs() + 0.1
    k[0, at, 0, 0] = float("-inf")
    got = run(q, k, v, do, dict(causal=True))
    keep = [j for j in range(T) if j != at]
    n = T - at - 1                                       # the queries after the key
    want = tk.attention(q[:, -n:], k[:, keep], v[:, keep], do[:, -n:], causal=True)
    for name in ("out", "dq"):
        value, tol = want[name]
        first = 1 if name == "dq" else 0
        tk.close(got[name][:, -n:, :, first:], value[..., first:], tol[..., first:], name)


def test_norm_sums_of_no_rows():
    """The gradients of the weights and the gate over no rows are zeros, by
    the C entry as by the binding."""
    C, G = 100, 3
    lib = _lib.load()
    need = ctypes.c_size_t()
    assert lib.mp3d_gated_norm_workspace_bytes(_lib.MP3D_F32, 0, C, G, ctypes.byref(need)) == 0
    w = torch.ones(C, device="cuda")
    gate = torch.ones(G, C, device="cuda")
    sums = [torch.full((n, C), float("nan"), device="cuda") for n in (G, 1, 1)]
    assert lib.mp3d_gated_norm_backward(
        None, None, None, None, gate.data_ptr(), w.data_ptr(), w.data_ptr(), None, None, None,
        *[t.data_ptr() for t in sums], _lib.MP3D_F32, 0, C, G, 1.0, _lib.MP3D_NORM_RMS, 3, 1e-6,
        None, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for t in sums:
        assert torch.equal(t, torch.zeros_like(t))
    e = torch.empty((0, C), device="cuda")
    how = dict(gate=gate, post_weight=w, pre_weight=w)
    _, _, stats = mp.mp3d_gated_norm_forward(e, e, **how)
    dx, dh, *got = mp.mp3d_gated_norm_backward(e, e, e, e, stats, **how)
    assert dx.shape == dh.shape == e.shape
    for t, like in zip(got, (gate, w, w)):
        assert torch.equal(t, torch.zeros_like(like))


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
def test_attention_training_under_graph_capture(dt):
    """Forward and backward with documents, a bias of near and then of far
    positions, a cap, and gradients of other sizes, captured once: every replay
    gives the eager bits."""
    T, H, D = 300, 4, 64
    docs = torch.tensor([[0, 90, 170, 300]], dtype=torch.int32, device="cuda")
    slopes = torch.full((H, 2), 0.05, device="cuda")
    pos = torch.zeros((2, 1, T), dtype=torch.int32, device="cuda")
    q, k, v, do = (torch.zeros((1, T, h, D), dtype=dt, device="cuda") for h in (H, 2, 2, H))

    def both():
        how = dict(causal=True, softcap=30.0, doc_offsets=docs, slopes=slopes, pos_q=pos,
                   pos_k=pos)
        out, lse = mp.mp3d_attention_forward(q, k, v, **how)
        return (out, lse) + mp.mp3d_attention_backward(do, q, k, v, out, lse, **how)

    cells = torch.stack((torch.arange(T) // 20, torch.arange(T) % 20)).int()[:, None].cuda()
    far = cells.clone()
    far[:, :, 170:] += 1 << 30
    inputs = []
    for n, (p, size) in enumerate(((cells, 1.0), (far, 2.0 ** -12), (cells, 2.0 ** 10))):
        ten = [t.cuda() for t in make(1, T, T, H, 2, D, dt, 90 + n)]
        inputs.append((p, ten[:3] + [(ten[3].float() * size).to(dt)]))

    def load(p, ten):
        pos.copy_(p)
        for t, new in zip((q, k, v, do), ten):
            t.copy_(new)

    want = []
    for p, ten in inputs:
        load(p, ten)
        want.append([t.clone() for t in both()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for rep in range(3):
        for (p, ten), ref in zip(inputs, want):
            load(p, ten)
            for t in got:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
            both()                                       # eager work between the replays
            torch.cuda.synchronize()
