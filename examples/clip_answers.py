"""Several answers about one clip, token by token, from one cache of the clip:
its keys and values are written once, in 8 or 4 bits or as they are, and every
answer's new tokens attend to them and to the answer's own cache.

    python examples/clip_answers.py [--dtype bfloat16] [--format e4m3] [--answers 8] [--new 6]

The block is that of token_block.py; nothing of the clip is kept per answer.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import token_block as tb  # noqa: E402

mp = tb.mp


class Caches:
    """A cache of the clip, shared, and one of each answer's tokens."""

    def __init__(self, clip_tokens, answers, new, dtype, device, format):
        self.format, shape = format, (tb.KEY_HEADS, tb.D)
        if format is None:
            make = lambda B, T: tuple(torch.zeros((B, T) + shape, dtype=dtype,  # noqa: E731
                                                  device=device) for _ in range(2))
        else:
            make = lambda B, T: mp.mp3d_cache_empty(B, T, *shape, format,  # noqa: E731
                                                    device=device)
        self.clip, self.own = make(1, clip_tokens), make(answers, new)
        self.lengths = torch.zeros(answers, dtype=torch.int32, device=device)

    def write(self, cache, k, v, start=None):
        if self.format is not None:
            mp.mp3d_cache_write(k, v, cache, self.format, start=start)
            return
        rows = torch.arange(k.shape[1], device=k.device) + (0 if start is None
                                                            else start.long()[:, None])
        at = torch.arange(k.shape[0], device=k.device)[:, None]
        cache[0][at, rows], cache[1][at, rows] = k, v


def answer(block, t, grid, tokens, format):
    """The block's sums (S, n, C) for the tokens (S, n, C) of S answers that
    follow the clip t (1, P, C) of a grid."""
    S, n, _ = tokens.shape
    caches = Caches(t.shape[1], S, n, t.dtype, t.device, format)
    _, z, _ = mp.mp3d_gated_norm_forward(t, pre_weight=block.first)
    _, k, v = block.project(z)
    k = mp.mp3d_rope_forward(k, None, block.inv_freq, tb.PAIRS, grid=grid)
    caches.write(caches.clip, k, v)
    out = []
    for i in range(n):
        x = tokens[:, i:i + 1].contiguous()
        _, z, _ = mp.mp3d_gated_norm_forward(x, pre_weight=block.first)
        q, k, v = block.project(z)
        # behind the clip on the first axis
        at = torch.tensor([grid[0] + i, 0, 0], dtype=torch.int32, device=t.device)
        q, k = mp.mp3d_rope_forward(q, k, block.inv_freq, tb.PAIRS,
                                    positions=at[:, None, None].expand(3, S, 1).contiguous())
        caches.write(caches.own, k, v, caches.lengths)
        caches.lengths += 1
        o, _ = mp.mp3d_attention_cached(q, caches.own, caches.clip, format=format,
                                        softcap=tb.CAP, kv_len=caches.lengths)
        h = o.view(x.shape) @ block.wo
        out.append(mp.mp3d_gated_norm_forward(x, h, gate=block.gate, post_weight=block.post,
                                              pre_weight=block.pre)[0])
    return torch.cat(out, 1)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--dtype", default="bfloat16", choices=("float32", "float16", "bfloat16"))
    p.add_argument("--format", default="e4m3", choices=("e4m3", "e2m1"))
    p.add_argument("--answers", type=int, default=8)
    p.add_argument("--new", type=int, default=6)
    a = p.parse_args(argv)
    dtype, dev = getattr(torch, a.dtype), torch.device("cuda")
    block = tb.Block(dtype, dev)
    g = torch.Generator().manual_seed(2)
    C = tb.HEADS * tb.D
    clip = torch.randn((1, C, 8, 28, 28), generator=g).to(dev, dtype)
    pooled, _ = mp.mp3d_forward(clip, 2, 2)
    t, grid = tb.tokens_of(pooled), tuple(pooled.shape[2:])
    tokens = torch.randn((a.answers, a.new, C), generator=g).to(dev, dtype)
    plain, few = answer(block, t, grid, tokens, None), answer(block, t, grid, tokens, a.format)
    far = (few.float() - plain.float()).norm() / plain.float().norm()
    print("%d answers of %d tokens about %d: %s off plain caches by %.2g"
          % (a.answers, a.new, t.shape[1], a.format, far))
    return plain, few, far.item()


if __name__ == "__main__":
    main()
