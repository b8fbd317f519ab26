"""Rotary positions over three axes against the float64 form: types, pair
layouts, head layouts, widths that no vector divides, positions far out,
in place, the backward as the transpose."""
import pytest
import torch

import _tokens as tk
import bwd_max_pool3d_amd as mp

pytestmark = pytest.mark.gpu

# (B, T or grid, Hq, Hk, D, pairs, interleaved)
CASES = [
    (1, 1, 1, 0, 2, (1, 0, 0), False),
    (32, 1, 16, 4, 128, (16, 24, 24), False),
    (2, (3, 5, 7), 4, 4, 64, (8, 12, 12), False),
    (2, (3, 5, 7), 4, 1, 64, (8, 12, 12), True),
    (3, 17, 5, 3, 80, (8, 12, 12), True),           # channels that do not turn
    (3, 17, 5, 3, 80, (8, 12, 12), False),
    (1, 33, 3, 2, 37, (5, 0, 6), False),             # odd channels
    (1, 33, 3, 2, 37, (5, 7, 6), True),
    (2, 9, 2, 2, 16, (0, 0, 0), False),              # nothing turns
    (1, (1, 1, 130), 1, 7, 96, (0, 48, 0), False),
    (2, 5, 1, 1, 1000, (100, 200, 200), False),      # more units than threads
    (1, 300, 6, 6, 20, (2, 4, 4), True),
]


def make(case, dt, seed):
    B, T, Hq, Hk, D, pairs, il = case
    grid = T if isinstance(T, tuple) else None
    n = grid[0] * grid[1] * grid[2] if grid else T
    q, k = tk.randn((B, n, Hq, D), seed, dt), tk.randn((B, n, Hk, D), seed + 1, dt)
    P = sum(pairs)
    f = torch.tensor([10000.0 ** (-i / max(P, 1)) for i in range(P)], dtype=torch.float32)
    if grid:
        t = torch.arange(n)
        cell = torch.stack((t // (grid[1] * grid[2]), t // grid[2] % grid[1], t % grid[2]))
        pos = cell[:, None].expand(3, B, n).contiguous().int()
    else:
        g = torch.Generator().manual_seed(seed + 2)
        pos = torch.randint(-1000, 100000, (3, B, n), generator=g, dtype=torch.int32)
    return q, k, f, pos, grid


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace(" ", "") for v in c))
@pytest.mark.parametrize("back", [False, True], ids=["forward", "backward"])
def test_rope(case, dt, back):
    B, T, Hq, Hk, D, pairs, il = case
    q, k, f, pos, grid = make(case, dt, 5)
    call = mp.mp3d_rope_backward if back else mp.mp3d_rope_forward
    how = dict(grid=grid) if grid else dict(positions=pos.cuda())
    got = call(q.cuda(), k.cuda() if Hk else None, f.cuda(), pairs, interleaved=il, **how)
    got = got if Hk else (got, None)
    for x, y, what in ((q, got[0], "q"), (k, got[1], "k")):
        if y is not None:
            want, tol = tk.rope(x, f, pairs, pos, il, -1.0 if back else 1.0)
            tk.close(y, want, tol, what)


@pytest.mark.parametrize("layout", ["qkv", "head_major", "misaligned", "expanded"])
@pytest.mark.parametrize("il", [False, True])
def test_layouts(layout, il):
    B, T, Hq, Hk, D, pairs, dt = 2, 29, 4, 2, 32, (4, 6, 6), torch.bfloat16
    q, k, f, pos, _ = make((B, T, Hq, Hk, D, pairs, il), dt, 7)
    if layout == "qkv":
        buf = torch.cat((q, k, q), 2).cuda()
        qd, kd = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hk]
    elif layout == "head_major":
        qd, kd = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (q, k))
    elif layout == "expanded":                       # one sequence for the whole batch
        q, k = q[:1].expand(B, -1, -1, -1), k[:1].expand(B, -1, -1, -1)
        qd, kd = q[:1].cuda().expand(B, -1, -1, -1), k[:1].cuda().expand(B, -1, -1, -1)
    else:                                            # rows start at odd elements
        qd, kd = (torch.nn.functional.pad(t, (1, 2)).cuda()[..., 1:1 + D] for t in (q, k))
    got = mp.mp3d_rope_forward(qd, kd, f.cuda(), pairs, positions=pos.cuda(), interleaved=il)
    for x, y in ((q, got[0]), (k, got[1])):
        tk.close(y, *tk.rope(x, f, pairs, pos, il))


def test_in_place_and_round_trip():
    """In place gives the same bits; the backward undoes the forward."""
    q, k, f, pos, _ = make((2, 21, 3, 3, 64, (8, 12, 12), False), torch.float32, 9)
    a = mp.mp3d_rope_forward(q.cuda(), k.cuda(), f.cuda(), (8, 12, 12), positions=pos.cuda())
    qd, kd = q.cuda(), k.cuda()
    b = mp.mp3d_rope_forward(qd, kd, f.cuda(), (8, 12, 12), positions=pos.cuda(), out=(qd, kd))
    assert b[0] is qd and torch.equal(a[0], qd) and torch.equal(a[1], kd)
    back = mp.mp3d_rope_backward(a[0], a[1], f.cuda(), (8, 12, 12), positions=pos.cuda())
    for x, y in ((q, back[0]), (k, back[1])):
        want, tol = tk.rope(x, f, (8, 12, 12), pos, False)
        # a turn keeps a pair's length: two passes, each within its bound
        tk.close(y, x.double(), 2 * tol.amax(-1, keepdim=True) + tol)


def test_gradient_against_differences():
    """The map is linear: a difference over any step is the derivative."""
    dt, pairs = torch.float32, (3, 4, 5)
    q, _, f, pos, _ = make((1, 7, 2, 0, 30, pairs, True), dt, 11)
    w, d = tk.randn(q.shape, 12, dt), tk.randn(q.shape, 13, dt)
    fwd = lambda x: mp.mp3d_rope_forward(x.cuda(), None, f.cuda(), pairs, positions=pos.cuda(),  # noqa: E731
                                         interleaved=True).cpu().double()
    grad = mp.mp3d_rope_backward(w.cuda(), None, f.cuda(), pairs, positions=pos.cuda(),
                                 interleaved=True).cpu().double()
    diff = ((fwd(q + d) - fwd(q - d)) * w.double()).sum() / 2
    step = ((q + d).double() - (q - d).double()) / 2
    size = (w.double().abs() * (q.double().abs() + d.double().abs())).sum() * 4
    assert abs(diff - (grad * step).sum()) <= 16 * tk.E * size


def test_empty():
    f = torch.ones(2, device="cuda")
    x = torch.empty((0, 3, 2, 8), device="cuda")
    assert mp.mp3d_rope_forward(x, None, f, (2, 0, 0), grid=(1, 1, 3)).shape == x.shape
    x = torch.empty((2, 0, 2, 8), device="cuda")
    p = torch.empty((3, 2, 0), dtype=torch.int32, device="cuda")
    assert mp.mp3d_rope_backward(x, None, f, (2, 0, 0), positions=p).shape == x.shape
