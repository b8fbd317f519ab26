"""The range of float16 in the attention backward: weights and their gradients
that leave it while the results do not."""
import pytest
import torch

import _tokens as tk
from test_gpu_attention import make, run

pytestmark = pytest.mark.gpu
F16 = torch.float16


def scaled(shape, seed, *size):
    return [(t.float() * s).to(F16) for t, s in zip(make(*shape, F16, seed), size)]


def check_f16(got, ten, how, monkeypatch):
    """tk.attention's bounds, but for weights and their gradients that keep
    float16's 11 bits however small they are.  What a rounding adds near 0:
    2^-37 to a weight (2^12 times it is rounded), and to a gradient e = p (do
    . v - delta) 2^-37 of a bound of |e| / 2, |do|_1 max |v| (2^15 or less is
    rounded); to a result 2^-25, its own type's."""
    q, k, v, do = ten
    most = float(do.double().abs().sum(-1).max() * v.double().abs().max())
    for names, tiny in ((("out", "dv"), 2.0 ** -37), (("dq", "dk"), 2.0 ** -37 * max(most, 1e-20))):
        monkeypatch.setitem(tk.TINY, F16, tiny)
        r = tk.attention(q, k, v, do, **how)
        for name in names:
            value, tol = r[name]
            assert value.abs().max() < 60000
            tk.close(got[name], value, tol + 2.0 ** -25, name)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_large_gradients(D, causal, monkeypatch):
    """Loss-scaled gradients: p (do . v - delta) passes float16, dq and dk do not."""
    ten = scaled((1, 70, 70, 2, 1, D), 70, 0.05, 0.05, 16.0, 4000.0)
    how = dict(causal=causal)
    if not causal:                                       # three keys a query: weights of a third
        how["doc_offsets"] = torch.arange(0, 71, 3, dtype=torch.int32)[None]
    check_f16(run(*ten, how), ten, how, monkeypatch)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qs,ks", [(2000.0, 2.0 ** -14), (2.0 ** -14, 2000.0)], ids=["dk", "dq"])
def test_small_gradients(qs, ks, D, monkeypatch):
    """Gradients near 2^-18 over 3000 keys: p (do . v - delta) near 1e-8,
    below float16's smallest step, dq (with large keys) or dk (with large
    queries) far above it."""
    ten = scaled((1, 300, 3000, 2, 1, D), 72, qs, ks, 1.0, 2.0 ** -18)
    check_f16(run(*ten, {}), ten, {}, monkeypatch)


@pytest.mark.parametrize("D", [64, 128])
def test_small_weights(D, monkeypatch):
    """100000 keys: weights near 1e-5, below float16's smallest normal number."""
    ten = scaled((1, 40, 100000, 1, 1, D), 71, 0.5, 0.5, 1.0, 30.0)
    check_f16(run(*ten, {}), ten, {}, monkeypatch)


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_unequal_size(D, monkeypatch):
    """Queries whose gradients differ by 2^20, in one block and between
    documents; queries without a gradient; a sequence without any."""
    ten = scaled((2, 200, 200, 2, 1, D), 73, 1.0, 1.0, 1.0, 1.0)
    size = torch.ones(2, 200, 1, 1)
    size[0, 50:100], size[0, 100:130], size[0, 130:] = 2.0 ** -10, 2.0 ** 10, 0.0
    size[1] = 0.0
    ten[3] = (ten[3].float() * size).to(F16)
    how = dict(causal=True, doc_offsets=torch.tensor([[0, 50, 100, 130, 200], [0, 9, 99, 199, 200]],
                                                     dtype=torch.int32))
    got = run(*ten, how)
    check_f16(got, ten, how, monkeypatch)
    for name in ("dq", "dk", "dv"):
        assert not got[name][1].any()


@pytest.mark.parametrize("Tq,Tk,Hq,Hk", [(1, 3000, 8, 2), (33, 17, 4, 1),
                                         (700, 40, 8, 1), (40, 700, 2, 2)])
def test_the_largest_value_wherever_it_stands(Tq, Tk, Hq, Hk, monkeypatch):
    """Shares of the keys of every size, the largest value in the first, the
    last or the middle key: its gradients do not leave the range."""
    for n, at in enumerate({0, Tk // 2, Tk - 1}):
        ten = scaled((2, Tq, Tk, Hq, Hk, 64), 82 + n, 0.05, 0.05, 1.0, 2000.0)
        ten[2][:, at] *= 64
        check_f16(run(*ten, {}), ten, {}, monkeypatch)
