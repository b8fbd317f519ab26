"""The token operators together, and what they share: graph capture, offsets
past 32 bits, tensors the binding refuses."""
import pytest
import torch

import _tokens as tk
import bwd_max_pool3d_amd as mp

pytestmark = pytest.mark.gpu


def block(x, w, grid, docs):
    """One pooled-volume block: pool, norm, rotary positions, attention, gated
    norm, and its backward, with every buffer given or kept."""
    y, idx = mp.mp3d_forward(x, 2, 2)
    B, C = y.shape[:2]
    t = y.flatten(2).transpose(1, 2).contiguous()          # (B, T, C)
    T = t.shape[1]
    _, z, s0 = mp.mp3d_gated_norm_forward(t, pre_weight=w["pre"])
    heads = z.view(B, T, 4, C // 4)
    q, k = mp.mp3d_rope_forward(heads, heads, w["freq"], w["pairs"], grid=grid)
    how = dict(softcap=10.0, doc_offsets=docs)
    o, lse = mp.mp3d_attention_forward(q, k, heads, **how)
    h = o.view(B, T, C)
    y2, z2, s1 = mp.mp3d_gated_norm_forward(t, h, gate=w["gate"], pre_weight=w["pre"])
    dx, dh, dgate, _, dpre = mp.mp3d_gated_norm_backward(None, z2, t, h, s1, gate=w["gate"],
                                                         pre_weight=w["pre"])
    dq, dk, dv = mp.mp3d_attention_backward(dh.view_as(o), q, k, heads, o, lse, **how)
    dq, dk = mp.mp3d_rope_backward(dq, dk, w["freq"], w["pairs"], grid=grid)
    dz = (dq + dk + dv).view(B, T, C)
    dt, _, _, _, _ = mp.mp3d_gated_norm_backward(dx, dz, t, None, s0, pre_weight=w["pre"])
    gy = dt.transpose(1, 2).contiguous().view_as(y)
    gx = mp.mp3d_backward(gy, idx, x.shape, kernel=2, stride=2, overlap=0)
    return y2, z2, gx, dgate, dpre


def setup(dt, seed):
    C = 64
    w = {"pre": tk.randn((C,), seed, dt, 0.1, 1.0).cuda(),
         "gate": tk.randn((2, C), seed + 1, dt, 0.5).cuda(), "pairs": (2, 3, 3),
         "freq": torch.tensor([100.0 ** (-i / 8) for i in range(8)], device="cuda")}
    x = tk.randn((2, C, 6, 10, 8), seed + 2, dt).cuda()
    docs = torch.tensor([[0, 20, 60], [0, 31, 55]], dtype=torch.int32, device="cuda")
    return x, w, (3, 5, 4), docs


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=tk.name_of)
def test_block_under_graph_capture(dt):
    """The whole block, captured once and replayed on new inputs, gives the
    eager bits on every replay."""
    x, w, grid, docs = setup(dt, 70)
    inputs = [tk.randn(x.shape, 80 + i, dt).cuda() for i in range(3)]
    refs = []
    for v in inputs:
        x.copy_(v)
        refs.append([t.clone() for t in block(x, w, grid, docs)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, w, grid, docs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block(x, w, grid, docs)
    torch.cuda.synchronize()
    for rep in range(2):
        for v, ref in zip(inputs, refs):
            x.copy_(v)
            for t in outs:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, ref):
                assert torch.equal(a, b)


def test_cache_past_32_bit_offsets():
    """Keys and values whose elements lie past 2^31: the strides of a long
    cache, over a buffer that is only touched where they point."""
    step, Tk, H, D = 1 << 23, 300, 2, 64                   # 300 rows, 2.5e9 elements apart in all
    buf = torch.empty(step * Tk, dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((1, Tk, H, D), (step * Tk, step, D, 1))
    v = buf.as_strided((1, Tk, H, D), (step * Tk, step, D, 1), 4096)
    kk, vv = (tk.randn((1, Tk, H, D), 90 + i, torch.bfloat16).cuda() for i in range(2))
    k.copy_(kk)
    v.copy_(vv)
    for Tq in (1, 150):
        q = tk.randn((1, Tq, 4, D), 92, torch.bfloat16).cuda()
        a = mp.mp3d_attention_forward(q, k, v, causal=True)
        b = mp.mp3d_attention_forward(q, kk, vv, causal=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ga = mp.mp3d_attention_backward(q, q, k, v, *a, causal=True)
        gb = mp.mp3d_attention_backward(q, q, kk, vv, *b, causal=True)
        for s, t in zip(ga, gb):
            assert torch.equal(s, t)
    f = torch.ones(8, device="cuda")
    pos = torch.arange(Tk, dtype=torch.int32, device="cuda").expand(3, 1, Tk).contiguous()
    a = mp.mp3d_rope_forward(k, v, f, (4, 2, 2), positions=pos)
    b = mp.mp3d_rope_forward(kk, vv, f, (4, 2, 2), positions=pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_past_32_bit_offsets():
    rows, C = (1 << 17) + 3, 16384                         # 2^31 elements and a few rows
    x = torch.zeros((rows, C), dtype=torch.bfloat16, device="cuda")
    h = torch.zeros_like(x)
    x[-5:] = tk.randn((5, C), 93, torch.bfloat16).cuda()
    h[-5:] = tk.randn((5, C), 94, torch.bfloat16).cuda()
    y, z, stats = mp.mp3d_gated_norm_forward(x, h)
    ys, zs, ss = mp.mp3d_gated_norm_forward(x[-5:].contiguous(), h[-5:].contiguous())
    assert torch.equal(y[-5:], ys) and torch.equal(z[-5:], zs) and torch.equal(stats[-5:], ss)
    dx, dh, _, _, _ = mp.mp3d_gated_norm_backward(x, h, x, h, stats)
    dxs, dhs, _, _, _ = mp.mp3d_gated_norm_backward(x[-5:].contiguous(), h[-5:].contiguous(),
                                                    x[-5:].contiguous(), h[-5:].contiguous(), ss)
    assert torch.equal(dx[-5:], dxs) and torch.equal(dh[-5:], dhs)


def test_binding_refusals():
    """What the binding itself refuses, and the library's codes through it."""
    x = torch.zeros((1, 4, 2, 8), device="cuda")
    f = torch.ones(4, device="cuda")
    bad = [
        (ValueError, lambda: mp.mp3d_rope_forward(x[0], x[0], f, (4, 0, 0), grid=(1, 1, 4))),
        (ValueError, lambda: mp.mp3d_rope_forward(x.transpose(2, 3), None, f, (4, 0, 0),
                                                  grid=(1, 1, 4))),
        (ValueError, lambda: mp.mp3d_rope_forward(x, x[:, :3], f, (4, 0, 0), grid=(1, 1, 4))),
        (ValueError, lambda: mp.mp3d_rope_forward(x, x.half(), f, (4, 0, 0), grid=(1, 1, 4))),
        (ValueError, lambda: mp.mp3d_rope_forward(x, x, f[:3], (4, 0, 0), grid=(1, 1, 4))),
        (ValueError, lambda: mp.mp3d_rope_forward(x, x, f, (4, 0, 0))),
        (TypeError, lambda: mp.mp3d_rope_forward(x.double(), None, f, (4, 0, 0), grid=(1, 1, 4))),
        (mp.Mp3dError, lambda: mp.mp3d_rope_forward(x, x, f, (4, 0, 0), grid=(1, 1, 5))),
        (ValueError, lambda: mp.mp3d_attention_forward(x, x, x[:, :3])),
        (ValueError, lambda: mp.mp3d_attention_forward(x, x, x.half())),
        (ValueError, lambda: mp.mp3d_attention_forward(x, x, x, kv_len=torch.ones(1))),
        (ValueError, lambda: mp.mp3d_attention_forward(x, x, x, slopes=f.view(2, 2))),
        (ValueError, lambda: mp.mp3d_attention_forward(x, x, x, pos_q=f)),
        (TypeError, lambda: mp.mp3d_attention_forward(x.double(), x.double(), x.double())),
        (mp.Mp3dError, lambda: mp.mp3d_attention_forward(x, x, x, prefix=torch.ones(
            1, dtype=torch.int32, device="cuda"))),
        (mp.Mp3dError, lambda: mp.mp3d_attention_forward(
            torch.zeros((1, 2, 1, 136), device="cuda"), *[torch.zeros((1, 2, 1, 136),
                                                                      device="cuda")] * 2)),
        (ValueError, lambda: mp.mp3d_gated_norm_forward(x.transpose(1, 2))),
        (ValueError, lambda: mp.mp3d_gated_norm_forward(x, x, norm="group")),
        (ValueError, lambda: mp.mp3d_gated_norm_forward(x, x.half())),
        (ValueError, lambda: mp.mp3d_gated_norm_forward(x, x, pre_weight=f)),
        (mp.Mp3dError, lambda: mp.mp3d_gated_norm_forward(x, x, gate=torch.zeros((3, 8),
                                                                                 device="cuda"))),
        (mp.Mp3dError, lambda: mp.mp3d_gated_norm_forward(x, pre_norm=False)),
        (ValueError, lambda: mp.mp3d_gated_norm_backward(x, None, x, x, f)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("dt,T,Hq,Hk,D", [(torch.float32, 520, 4, 2, 64),
                                          (torch.float32, 2049, 2, 1, 128),
                                          (torch.bfloat16, 4100, 2, 2, 72)], ids=str)
def test_long_chunks_of_few_heads(dt, T, Hq, Hk, D):
    """Many queries dealt out by chunks of keys give what the same queries
    give in a batch that fills the card."""
    q, k, v = (tk.randn((1, T, h, D), 95 + i, dt).cuda() for i, h in enumerate((Hq, Hk, Hk)))
    n = 128                                                 # workgroups: over 5/8 of the CUs
    how = dict(causal=True, softcap=20.0)
    a, la = mp.mp3d_attention_forward(q, k, v, **how)
    rep = [t.expand(n, -1, -1, -1) for t in (q, k, v)]
    b, lb = mp.mp3d_attention_forward(*rep, **how)
    # both are within the bounds of one result: out is a mean of |v| <= 6
    # deviations, its weights rounded (2^-9 for bfloat16), itself rounded
    # (2^-9), exponents off by the binary32 products' error (D 2^-24 of |s| <= 20)
    unit = 2.0 ** -9 if dt == torch.bfloat16 else 2.0 ** -24
    tol = 2 * (2 * unit + 20 * D * 2.0 ** -24) * 6
    assert (a.float() - b[0].float()).abs().max().item() <= tol
    assert (la - lb[0]).abs().max().item() <= 2 * 20 * D * 2.0 ** -24 + T * 2.0 ** -24
