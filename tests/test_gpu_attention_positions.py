"""Distances of positions anywhere in int32."""
import pytest
import torch

import _tokens as tk
from test_gpu_attention import check, make, run

pytestmark = pytest.mark.gpu

# int32 offsets of documents whose own cells are near each other
FAR = [0, (1 << 30) + 7, -(1 << 31) + 3, (1 << 31) - 70, -(1 << 25) - 1, 1 << 24]


def cells(starts, T, axes, far):
    """(axes, 1, T) positions: each document its own cells at its own offset,
    the axes at different ones; negative directions too."""
    pos = torch.zeros((axes, 1, T), dtype=torch.int64)
    for a in range(axes):
        for d, (s, e) in enumerate(zip(starts[:-1], starts[1:])):
            j = torch.arange(e - s)
            cell = (j // 12, j // 4 % 3, j % 4)[a]
            pos[a, 0, s:e] = far[(d + a) % len(far)] + cell
    assert int(pos.min()) >= -(1 << 31) and int(pos.max()) < 1 << 31
    return pos.int()


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Tq", [2, 60, 300])
def test_documents_at_far_positions(Tq, D, dt):
    """Tokens near each other, far from the sequence's first key, their
    documents far from one another and in one block of queries."""
    starts, axes = [0, 40, 90, 150, 240, 299, 300], 3
    pos = cells(starts, 300, axes, FAR)
    g = torch.Generator().manual_seed(61)
    how = dict(doc_offsets=torch.tensor([starts], dtype=torch.int32), pos_k=pos,
               pos_q=pos[:, :, 300 - Tq:].contiguous(), slopes=torch.rand((2, axes), generator=g))
    check(*make(1, Tq, 300, 2, 1, D, dt, 62), how)


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("Tq", [4, 200])
def test_far_distances(Tq, dt):
    """Positions over all of int32 that all see each other: distances up to
    2^32, to their 24 bits (slopes near 2^-27: biases up to 48)."""
    B, Tk, Hq, axes = 2, 200, 2, 3
    g = torch.Generator().manual_seed(63)
    draw = lambda n: torch.randint(-(1 << 31), 1 << 31, (axes, B, n), generator=g).int()  # noqa: E731
    pk = draw(Tk)
    pk[:, :, 0], pk[:, :, 1], pk[:, :, 2] = -(1 << 31), (1 << 31) - 1, 0
    how = dict(slopes=torch.rand((Hq, axes), generator=g) * 2.0 ** -27, pos_q=draw(Tq), pos_k=pk)
    check(*make(B, Tq, Tk, Hq, 1, 64, dt, 64), how)


@pytest.mark.parametrize("Tq", [3, 70])
def test_first_key_far_from_all(Tq):
    """Only the first key is far: the others' distances stay exact, in the
    forward and in the gradients, as if the first key were not there."""
    T = 70
    q, k, v, do = make(1, Tq, T, 2, 2, 64, torch.float32, 65)
    pos = (torch.arange(T) * 3 + (1 << 30)).int()[None, None]
    pos[0, 0, 0] = 0
    pos_q = (torch.arange(T - Tq, T) * 3 + (1 << 30)).int()[None, None]
    how = dict(slopes=torch.full((2, 1), 0.25), pos_k=pos, pos_q=pos_q)
    got = run(q, k, v, do, how)
    # (the first key's weight is exp(-2^28): none)
    want = tk.attention(q, k[:, 1:], v[:, 1:], do, slopes=how["slopes"], pos_q=pos_q - (1 << 30),
                        pos_k=pos[:, :, 1:] - (1 << 30))
    for name in ("out", "lse", "dq"):
        tk.close(got[name], *want[name], name)
    for name in ("dk", "dv"):
        tk.close(got[name][:, 1:], *want[name], name)
        assert torch.equal(got[name][:, :1].cpu(), torch.zeros_like(k[:, :1]))
