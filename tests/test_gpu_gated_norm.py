"""The gated norm and its backward against the float64 form: types, widths
of every kernel variant, parts left out, gates per channel and per batch."""
import pytest
import torch

import _tokens as tk
import bwd_max_pool3d_amd as mp

pytestmark = pytest.mark.gpu


def make(rows, C, gates, dt, seed, post=True, pre=True):
    t = {"x": tk.randn((rows, C), seed, dt), "h": tk.randn((rows, C), seed + 1, dt, 2.0, 0.5),
         "gate": tk.randn((gates, C), seed + 2, dt, 0.5) if gates else None,
         "post": tk.randn((C,), seed + 3, dt, 0.1, 1.0) if post else None,
         "pre": tk.randn((C,), seed + 4, dt, 0.1, 1.0) if pre else None,
         "dy": tk.randn((rows, C), seed + 5, dt), "dz": tk.randn((rows, C), seed + 6, dt)}
    return t


def dev(v):
    return None if v is None else v.cuda()


def check(t, rs, kind, eps=1e-6, post_norm=True, pre_norm=True, h=True, dy=True):
    x, hh = t["x"], t["h"] if h else None
    gate, post = (t["gate"], t["post"]) if h else (None, None)
    pre = t["pre"] if pre_norm else None
    dz = t["dz"] if pre_norm else None
    dyt = t["dy"] if dy else None
    how = dict(gate=dev(gate), post_weight=dev(post), pre_weight=dev(pre), residual_scale=rs,
               norm=kind, eps=eps, post_norm=post_norm, pre_norm=pre_norm)
    y, z, stats = mp.mp3d_gated_norm_forward(x.cuda(), dev(hh), **how)
    g = mp.mp3d_gated_norm_backward(dev(dyt), dev(dz), x.cuda(), dev(hh), stats, **how)
    want = tk.gated_norm(x, hh, gate, post, pre, rs, kind == "layer", eps, post_norm and h,
                         pre_norm, dyt, dz, grads=True)
    got = {"y": y, "z": z}
    got.update(zip(("dx", "dh", "dgate", "dpost", "dpre"), g))
    for name, (value, tol) in want.items():
        tk.close(got[name], value, tol, name)
    for name, v in got.items():
        if name not in want and name != "y":
            assert v is None, name


# every kernel variant: 64, 256 and 1024 threads a row, 8 and 16 elements a
# thread, whole vectors and single elements
WIDTHS = [1, 7, 64, 255, 512, 520, 1000, 1001, 1024, 1032, 2048, 2049, 4096, 4100, 8192, 8193,
          16384]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(C, dt, kind):
    rows = 6 if C > 2000 else 13
    check(make(rows, C, 1, dt, 20), 0.5, kind)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,gates", [(1, 0), (1, 1), (5, 5), (12, 3), (1500, 1), (1600, 800),
                                        (2000, 2000), (4096, 4), (3000, 1500), (777, 0)])
def test_rows_and_gates(rows, gates, kind):
    """Groups of every size: one row each, fewer and more groups than
    workgroups, no gate."""
    check(make(rows, 40, gates, torch.float32, 21), 1.25, kind)
    check(make(rows, 40, gates, torch.bfloat16, 22), 1.25, kind)


@pytest.mark.parametrize("rows,C,gates", [(300, 2000, 2), (900, 1100, 900), (40, 6000, 2),
                                          (300, 5000, 300)])
def test_wide_rows_and_gates(rows, C, gates):
    check(make(rows, C, gates, torch.float16, 23), 0.75, "layer")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("how", [dict(post_norm=False), dict(pre_norm=False), dict(h=False),
                                 dict(post_norm=False, pre_norm=False), dict(dy=False),
                                 dict(pre_norm=False, dy=True)], ids=str)
@pytest.mark.parametrize("C", [96, 1500])
def test_parts(how, kind, C):
    for dt in tk.TYPES:
        check(make(37, C, 1, dt, 24), 0.5, kind, **how)
        check(make(37, C, 0, dt, 25, post=False, pre=False), 0.5, kind, **how)


def test_large_mean_and_constant_rows():
    """The mean is taken before the squares: a mean of 1000 deviations does
    not drown them; a constant row has n = 0 (eps keeps it finite)."""
    t = make(9, 300, 1, torch.float32, 26)
    t["h"] = t["h"] + 2000.0
    t["x"][3] = 0.25
    t["h"][3] = 7.0
    check(t, 0.5, "layer", eps=1e-5)


def test_nan_stays_in_its_row():
    t = make(8, 200, 1, torch.bfloat16, 27)
    t["h"][5, 17] = float("nan")
    y, z, _ = mp.mp3d_gated_norm_forward(t["x"].cuda(), t["h"].cuda(), gate=t["gate"].cuda())
    bad = torch.isnan(y).any(1) | torch.isnan(z).any(1)
    assert bad.tolist() == [i == 5 for i in range(8)]


def test_shapes_empty_and_preallocated():
    x = tk.randn((2, 5, 48), 28, torch.float16).cuda()
    h = tk.randn((2, 5, 48), 29, torch.float16).cuda()
    out = (torch.empty_like(x), torch.empty_like(x))
    y, z, stats = mp.mp3d_gated_norm_forward(x, h, out=out)
    assert y is out[0] and z is out[1] and stats.shape == (10, 4)
    flat = mp.mp3d_gated_norm_forward(x.view(10, 48), h.view(10, 48))
    assert torch.equal(flat[0].view_as(y), y) and torch.equal(flat[1].view_as(z), z)
    e = torch.empty((0, 48), device="cuda")
    w = torch.ones(48, device="cuda")
    y, z, stats = mp.mp3d_gated_norm_forward(e, e, pre_weight=w)
    g = mp.mp3d_gated_norm_backward(e, e, e, e, stats, pre_weight=w)
    assert y.shape == e.shape and torch.equal(g[4], torch.zeros_like(w))


def test_gradient_against_differences():
    """<gradient, direction> against a central difference of the forward.  The
    step is 2^-6 of the inputs' size: its square (the difference's own error,
    through third derivatives of order one) is 2.4e-4, and float32's error
    over the step about 1e-5, both of the size of |gradient| |direction|."""
    for kind in ("rms", "layer"):
        t = make(6, 50, 1, torch.float32, 30)
        how = lambda t: dict(gate=dev(t["gate"]), post_weight=dev(t["post"]),  # noqa: E731
                             pre_weight=dev(t["pre"]), residual_scale=0.5, norm=kind)

        def loss(t):
            y, z, _ = mp.mp3d_gated_norm_forward(t["x"].cuda(), t["h"].cuda(), **how(t))
            return ((y.double().cpu() * t["dy"].double()).sum()
                    + (z.double().cpu() * t["dz"].double()).sum())

        _, _, stats = mp.mp3d_gated_norm_forward(t["x"].cuda(), t["h"].cuda(), **how(t))
        g = mp.mp3d_gated_norm_backward(t["dy"].cuda(), t["dz"].cuda(), t["x"].cuda(),
                                        t["h"].cuda(), stats, **how(t))
        for name, grad in zip(("x", "h", "gate", "post", "pre"), g):
            d = tk.randn(t[name].shape, 31, torch.float32)
            up, down = dict(t), dict(t)
            up[name], down[name] = t[name] + d / 64, t[name] - d / 64
            diff = (loss(up) - loss(down)) * 32
            step = (up[name].double() - down[name].double()) * 32
            grad = grad.cpu().double()
            assert abs(diff - (grad * step).sum()) <= 1e-3 * grad.norm() * step.norm(), name
