"""Caps at the ends of their range, scales far from 1 beside them, and both of
the forms in which 16-bit types take the tanh."""
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


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("shape", [(1, 4, 400, 4, 2, 64), (2, 200, 200, 2, 1, 64),
                                   (1, 300, 300, 2, 2, 128)], ids=str)
@pytest.mark.parametrize("cap", [0.5, 2.0, 20.0, 50.0])
@pytest.mark.parametrize("causal", [False, True])
def test_both_forms_of_the_tanh(causal, cap, shape, dt):
    """Scores of up to about 5: beyond a cap of 0.5, near 2's quarter, all
    within the others'."""
    check(*make(*shape, dt, 78), dict(softcap=cap, causal=causal))


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("part", [0.2499, 0.2501, 0.5])
def test_scores_around_a_quarter_of_the_cap(part, dt):
    """One query and key whose score alone reaches `part` of the cap, the other
    scores far below: the wave's tiles go by either form."""
    cap = 40.0
    q, k, v, do = make(1, 96, 96, 1, 1, 64, dt, 79)
    q, k = (q.float() * 0.3).to(dt), (k.float() * 0.3).to(dt)
    q[0, 10, 0], k[0, 20, 0] = 0, 0
    q[0, 10, 0, 5], k[0, 20, 0, 5] = 16.0, part * cap * 8 / 16.0
    check(q, k, v, do, dict(softcap=cap))


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e4], ids=str)
@pytest.mark.parametrize("Tq", [2, 180])
def test_what_is_masked_changes_no_bit_under_a_cap(value, Tq, dt):
    """Scores far below the cap, and a key that is not, seen by some queries:
    the others keep every bit."""
    Tk, at = 180, 179 if Tq == 2 else 101
    q, k, v, do = make(1, Tq, Tk, 4, 2, 64, dt, 80)
    how = dict(causal=True, softcap=50.0)
    clean = run(q, k, v, do, how)
    k[0, at, :, 5] = value
    got = run(q, k, v, do, how)
    see = at - (Tk - Tq)                                 # the first query that sees that key
    for name in ("out", "dq"):
        assert torch.equal(got[name][:, :see], clean[name][:, :see]), name
    assert torch.equal(got["lse"][:, :, :see], clean["lse"][:, :, :see])
