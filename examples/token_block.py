"""A block of tokens over a pooled volume, as a user would put it together:
clips are pooled, every cell becomes a token, and a pre-norm attention block
with rotary positions, capped scores and a gated residual runs over them;
first a training pass (forward and backward), then new tokens one at a time
from a cache of the clip's keys and values.

    python examples/token_block.py [--dtype bfloat16] [--steps 20] [--new 8]

Projections are plain matrix products; everything else is this library's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_max_pool3d_amd as mp  # noqa: E402

HEADS, KEY_HEADS, D = 8, 2, 64
PAIRS = (8, 12, 12)                       # rotary pairs on the axes (depth, height, width)
CAP = 30.0


class Block:
    """Weights of one block of ``HEADS`` heads that share ``KEY_HEADS``."""

    def __init__(self, dtype, device, seed=0):
        g = torch.Generator().manual_seed(seed)
        C = HEADS * D

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g) * scale).to(device=device, dtype=dtype)

        self.wq = normal(C, C, scale=C ** -0.5)
        self.wk = normal(C, KEY_HEADS * D, scale=C ** -0.5)
        self.wv = normal(C, KEY_HEADS * D, scale=C ** -0.5)
        self.wo = normal(C, C, scale=C ** -0.5)
        self.first = 1 + normal(C, scale=0.1)           # norm before attention
        self.post = 1 + normal(C, scale=0.1)            # norm of its result
        self.pre = 1 + normal(C, scale=0.1)             # norm before what follows
        self.gate = normal(1, C, scale=0.5)
        self.inv_freq = torch.tensor([100.0 ** (-i / n) for n in PAIRS for i in range(n)],
                                     dtype=torch.float32, device=device)

    def project(self, z):
        B, T, _ = z.shape
        return ((z @ self.wq).view(B, T, HEADS, D), (z @ self.wk).view(B, T, KEY_HEADS, D),
                (z @ self.wv).view(B, T, KEY_HEADS, D))

    def forward(self, t, grid):
        """(B, T, C) tokens of a grid: the block's sum and its norm, and what
        the backward and a cache need."""
        _, z, s0 = mp.mp3d_gated_norm_forward(t, pre_weight=self.first)
        q, k, v = self.project(z)
        q, k = mp.mp3d_rope_forward(q, k, self.inv_freq, PAIRS, grid=grid)
        o, lse = mp.mp3d_attention_forward(q, k, v, softcap=CAP, causal=True)
        h = o.view(t.shape) @ self.wo
        y, zn, s1 = mp.mp3d_gated_norm_forward(t, h, gate=self.gate, post_weight=self.post,
                                               pre_weight=self.pre)
        return y, zn, (t, z, q, k, v, o, lse, h, s0, s1)

    def backward(self, dy, dz, kept, grid):
        """Gradient of the tokens (the weights' products are left out but for
        the norms', which come with it)."""
        t, z, q, k, v, o, lse, h, s0, s1 = kept
        dt, dh, dgate, dpost, dpre = mp.mp3d_gated_norm_backward(
            dy, dz, t, h, s1, gate=self.gate, post_weight=self.post, pre_weight=self.pre)
        do = (dh @ self.wo.t()).view_as(o)
        dq, dk, dv = mp.mp3d_attention_backward(do, q, k, v, o, lse, softcap=CAP, causal=True)
        dq, dk = mp.mp3d_rope_backward(dq, dk, self.inv_freq, PAIRS, grid=grid)
        dz0 = (dq.flatten(2) @ self.wq.t() + dk.flatten(2) @ self.wk.t()
               + dv.flatten(2) @ self.wv.t())
        dt, _, _, _, dfirst = mp.mp3d_gated_norm_backward(dt, dz0, t, None, s0,
                                                          pre_weight=self.first)
        return dt, (dgate, dpost, dpre, dfirst)

    def step(self, t, positions, kc, vc, lengths):
        """One new token of each sequence (B, 1, C): its key and value go into
        the caches at ``lengths``, which are raised by one."""
        _, z, _ = mp.mp3d_gated_norm_forward(t, pre_weight=self.first)
        q, k, v = self.project(z)
        q, k = mp.mp3d_rope_forward(q, k, self.inv_freq, PAIRS, positions=positions)
        rows = torch.arange(t.shape[0], device=t.device)
        kc[rows, lengths.long()] = k[:, 0]
        vc[rows, lengths.long()] = v[:, 0]
        lengths += 1
        o, _ = mp.mp3d_attention_forward(q, kc, vc, softcap=CAP, causal=True, kv_len=lengths)
        h = o.view(t.shape) @ self.wo
        return mp.mp3d_gated_norm_forward(t, h, gate=self.gate, post_weight=self.post,
                                          pre_weight=self.pre)[:2]


def tokens_of(pooled):
    """(B, C, D, H, W) -> (B, D H W, C)."""
    return pooled.flatten(2).transpose(1, 2).contiguous()


def train_pass(block, clips):
    """Pool, block and the gradient of the clips under a sum of squares."""
    pooled, idx = mp.mp3d_forward(clips, 2, 2)
    grid, t = pooled.shape[2:], tokens_of(pooled)
    y, zn, kept = block.forward(t, grid)
    dt, _ = block.backward(y, zn, kept, grid)            # of (|y|^2 + |z|^2) / 2
    gp = dt.transpose(1, 2).contiguous().view_as(pooled)
    return y, kept, mp.mp3d_backward(gp, idx, clips.shape, kernel=2, stride=2, overlap=0)


def decode(block, t, grid, known):
    """The tokens of t from ``known`` on, one at a time: what step gives."""
    B, T, _ = t.shape
    kc, vc = (torch.zeros((B, T, KEY_HEADS, D), dtype=t.dtype, device=t.device) for _ in range(2))
    where = torch.arange(T, device=t.device)
    w, hw = grid[2], grid[1] * grid[2]
    pos = torch.stack((where // hw, where % hw // w, where % w)).to(torch.int32)
    # the clip's own tokens, at their cells of the grid
    _, z, _ = mp.mp3d_gated_norm_forward(t[:, :known].contiguous(), pre_weight=block.first)
    q, k, v = block.project(z)
    _, k = mp.mp3d_rope_forward(q, k, block.inv_freq, PAIRS,
                                positions=pos[:, None, :known].expand(-1, B, -1).contiguous())
    kc[:, :known], vc[:, :known] = k, v
    lengths = torch.full((B,), known, dtype=torch.int32, device=t.device)
    return torch.cat([block.step(t[:, i:i + 1].contiguous(),
                                 pos[:, None, i:i + 1].expand(-1, B, -1).contiguous(), kc, vc,
                                 lengths)[0] for i in range(known, T)], 1)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--dtype", default="bfloat16", choices=("float32", "float16", "bfloat16"))
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--new", type=int, default=8)
    a = p.parse_args(argv)
    dtype, dev = getattr(torch, a.dtype), torch.device("cuda")
    block = Block(dtype, dev)
    g = torch.Generator().manual_seed(1)
    clips = torch.randn((2, HEADS * D, 8, 28, 28), generator=g).to(dev, dtype)
    y, kept, gx = train_pass(block, clips)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        train_pass(block, clips)
    end.record()
    torch.cuda.synchronize()
    print("pool, block and gradient of %s: %.2f ms, |gx| %.4g"
          % (tuple(clips.shape), start.elapsed_time(end) / max(a.steps, 1), gx.float().norm()))
    t, T = kept[0], y.shape[1]
    some = decode(block, t, (4, 14, 14), T - a.new)
    far = (some.float() - y[:, T - a.new:].float()).norm() / y[:, T - a.new:].float().norm()
    print("%d tokens from the cache: relative difference from the whole pass %.2g" % (a.new, far))
    return y, gx, far.item()


if __name__ == "__main__":
    main()
