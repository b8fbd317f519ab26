"""The example's block: gradients of its norms' weights and its gate are those
of the parameters, summed over all tokens that share them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_gradients_have_the_parameters_shapes():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "token_block.py")
    spec = importlib.util.spec_from_file_location("token_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    block = example.Block(torch.float32, "cuda")
    g = torch.Generator().manual_seed(81)
    t, dy, dz = (torch.randn((3, 24, example.HEADS * example.D), generator=g).cuda()
                 for _ in range(3))
    *_, kept = block.forward(t, (2, 3, 4))
    _, grads = block.backward(dy, dz, kept, (2, 3, 4))
    for got, like in zip(grads, (block.gate, block.post, block.pre, block.first)):
        assert got.shape == like.shape
    # the gate's, by its formula: sum of dy + n_y^T(pre dz) times post n(h)
    h, s1 = kept[7].double(), kept[9].view(3, 24, 4).double()
    n = h * s1[..., 1:2]                                 # (RMS: no mean)
    y = t.double() + block.gate.double() * block.post.double() * n
    ny = y * s1[..., 3:4]
    d = block.pre.double() * dz.double()
    dyt = dy.double() + s1[..., 3:4] * (d - ny * (d * ny).mean(-1, keepdim=True))
    want = (dyt * block.post.double() * n).sum((0, 1))
    # 72 rows of terms within 2^-18 of their size (statistics in binary32 over 512 channels)
    size = (dyt * block.post.double() * n).abs().sum((0, 1))
    assert ((grads[0][0].double() - want).abs() <= 2.0 ** -18 * size).all()
