"""The example of several answers about one clip runs, and with plain caches
gives what a cache of clip and answer together gives, answer by answer."""
import importlib.util
import os
import sys

import pytest
import torch

import bwd_max_pool3d_amd as mp

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    path = os.path.join(HERE, "examples", "clip_answers.py")
    spec = importlib.util.spec_from_file_location("clip_answers", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_runs(dtype, fmt):
    plain, few, far = load().main(["--dtype", dtype, "--format", fmt, "--answers", "5", "--new", "3"])
    assert plain.shape == few.shape == (5, 3, 512)
    assert torch.isfinite(plain).all() and torch.isfinite(few).all() and far > 0


@pytest.mark.parametrize("dtype,unit", [("float32", 2.0 ** -24), ("float16", 2.0 ** -11),
                                        ("bfloat16", 2.0 ** -8)])
def test_plain_caches_agree_with_one_cache(dtype, unit):
    example = load()
    tb, dt, dev = example.tb, getattr(torch, dtype), torch.device("cuda")
    block = tb.Block(dt, dev)
    g = torch.Generator().manual_seed(3)
    C, S, n, grid = tb.HEADS * tb.D, 4, 3, (2, 7, 9)
    P = grid[0] * grid[1] * grid[2]
    t = torch.randn((1, P, C), generator=g).to(dev, dt)
    tokens = torch.randn((S, n, C), generator=g).to(dev, dt)
    got = example.answer(block, t, grid, tokens, None)
    # the block's own step, with a cache of the clip for every answer
    kc, vc = (torch.zeros((S, P + n, tb.KEY_HEADS, tb.D), dtype=dt, device=dev) for _ in range(2))
    _, z, _ = mp.mp3d_gated_norm_forward(t, pre_weight=block.first)
    _, k, v = block.project(z)
    k = mp.mp3d_rope_forward(k, None, block.inv_freq, tb.PAIRS, grid=grid)
    kc[:, :P], vc[:, :P] = k, v
    lengths = torch.full((S,), P, dtype=torch.int32, device=dev)
    want = []
    for i in range(n):
        at = torch.tensor([grid[0] + i, 0, 0], dtype=torch.int32, device=dev)
        pos = at[:, None, None].expand(3, S, 1).contiguous()
        want.append(block.step(tokens[:, i:i + 1].contiguous(), pos, kc, vc, lengths)[0])
    want = torch.cat(want, 1).float()
    far = (got.float() - want).norm() / want.norm()
    # o, h and y are rounded apart in the two ways: sqrt(2 * 3) roundings in all;
    # binary32 sums of up to 512 terms differ by up to sqrt(512) units
    few = 6 ** 0.5 * unit
    assert far <= (few if dtype != "float32" else few * 512 ** 0.5)
    assert "token_block" in sys.modules
