"""Caps at the ends of their range, and scales far from 1 beside them."""
import pytest
import torch

import _tokens as tk
from test_gpu_attention import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("shape", [(1, 3, 90, 2, 1, 64), (1, 90, 90, 2, 1, 64)], ids=str)
@pytest.mark.parametrize("cap", [1e-4, 1e-8, 1e-12, 1e-20, 1e-30])
def test_small_caps(cap, shape, dt):
    """A cap far below the scores: all weights alike, a query of zeros too."""
    q, k, v, do = make(*shape, dt, 67)
    q[:, 1], k[:, 5] = 0, 0
    got = run(q, k, v, do, dict(softcap=cap))
    want = tk.attention(q, k, v, do, softcap=cap)
    for name in ("out", "lse", "dv"):
        tk.close(got[name], *want[name], name)
    for name in ("dq", "dk"):
        assert torch.isfinite(got[name]).all(), name


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=tk.name_of)
@pytest.mark.parametrize("cap", [1e15, 1e30])
@pytest.mark.parametrize("scale", [1e-25, 1e-3, None, 1e3])
def test_large_caps(cap, scale, dt):
    """A cap far above the scores changes nothing."""
    q, k, v, do = make(1, 90, 90, 2, 1, 64, dt, 68)
    size = 1.0 if scale is None else (8 * scale) ** -0.5
    q, k = (q.float() * size).to(dt), (k.float() * size).to(dt)
    check(q, k, v, do, dict(softcap=cap, scale=scale))


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("Tq", [3, 90])
@pytest.mark.parametrize("cap", [1e-8, 1e-30])
def test_scores_of_zero_under_a_small_cap(cap, Tq, dt):
    """All scores 0: all weights alike, and dq = scale sum_j e_ij k_j."""
    q, k, v, do = make(1, Tq, 90, 2, 1, 64, dt, 69)
    check(torch.zeros_like(q), k, v, do, dict(softcap=cap))
