"""Caches in 8 and 4 bits on the GPU: codes, scales and values are the plain
form's bit for bit, and nothing else is written."""
import pytest
import torch

import _caches as oracle
import _tokens as tk
import bwd_max_pool3d_amd as mp

pytestmark = pytest.mark.gpu

FMT = oracle.FORMATS


def empty(B, T, H, D, fmt, fill=0xA5):
    c = mp.mp3d_cache_empty(B, T, H, D, fmt)
    for t in c:
        t.fill_(fill)
    return c


def same(got, want, what=""):
    """Equal bit for bit, any NaN for a NaN."""
    got = got.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape, what
    if got.dtype != torch.uint8:
        nan = torch.isnan(want)
        assert torch.equal(nan, torch.isnan(got)), "%s: NaN elsewhere" % what
        got, want = (torch.where(nan, torch.zeros_like(t), t) for t in (got, want))
        assert torch.equal(torch.signbit(got), torch.signbit(want)), "%s: signs" % what
    off = (got != want).nonzero()
    assert len(off) == 0, "%s: %d differ, the first at %s: %s, not %s" % (
        what, len(off), off[0].tolist(), got[tuple(off[0])], want[tuple(off[0])])


def values(B, T, H, D, dt, seed):
    """Groups of all magnitudes of the type, zeros, numbers halfway between
    codes, and the type's largest."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, T, H, D), generator=g)
    low, high = (-24, 15) if dt == torch.float16 else (-126, 127)
    e = torch.randint(low, high, (B, T, H, (D + 31) // 32), generator=g).float()
    x = (x * torch.exp2(e).repeat_interleave(32, -1)[..., :D].clamp(max=2.0 ** 126)).to(dt)
    # quarters and eighths of a power of two: many ties
    ties = torch.randint(-64, 65, (B, T, H, D), generator=g).to(dt)
    x = torch.where(torch.rand((B, T, H, 1), generator=g) < 0.4, ties, x)
    x = torch.where(torch.rand((B, T, H, 1), generator=g) < 0.1, torch.zeros_like(x), x)
    top = torch.finfo(dt).max
    x[0, 0, 0] = top
    x[0, 0, -1, 0] = -top
    x[-1, -1, 0] = torch.finfo(dt).smallest_normal / 4         # a subnormal
    return x


def check(k, v, fmt, cache, start, count, before=0xA5):
    """The cache holds these tokens at these rows, and what it held elsewhere."""
    B, T, H, D = k.shape
    rows = cache[0].shape[1]
    for i, x in enumerate((k, v)):
        codes, scales = oracle.write(x, fmt)
        for got, want in ((cache[2 * i], codes), (cache[2 * i + 1], scales)):
            full = torch.full(got.shape, before, dtype=torch.uint8)
            for b in range(B):
                s, n = int(start[b]), T if count is None else min(T, int(count[b]))
                for t in range(n):
                    if 0 <= s + t < rows:
                        full[b, s + t] = want[b, t]
            same(got, full, "part %d" % i)


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("D", [1, 7, 8, 31, 32, 33, 64, 72, 80, 96, 100, 128, 130, 1024])
def test_write_and_read(D, fmt, dt):
    B, T, H = (3, 5, 3) if D < 1000 else (1, 2, 2)
    k, v = values(B, T, H, D, dt, D), values(B, T, H, D, dt, D + 1)
    cache = empty(B, 9, H, D, fmt)
    start = torch.tensor([2, 0, 4][:B], dtype=torch.int32)
    mp.mp3d_cache_write(k.cuda(), v.cuda(), cache, fmt, start=start.cuda())
    check(k, v, fmt, cache, start, None)
    back = mp.mp3d_cache_read(cache, fmt, D, dt, rows=T, start=start.cuda())
    for got, x in zip(back, (k, v)):
        same(got, oracle.read(*oracle.write(x, fmt), fmt, D, dt), "values")
        assert torch.isfinite(got).all()                  # never past the type that was written


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("D", [33, 64])
def test_every_code_and_scale(D, fmt, dt):
    """Rows of random bytes: 255 and 0 among the scales, NaN among the codes,
    values past the type that is read."""
    B, T, H = 2, 300, 2
    g = torch.Generator().manual_seed(D)
    width, groups = oracle.widths(fmt, D)
    host = [torch.randint(0, 256, (B, T, H, n), generator=g).to(torch.uint8)
            for n in (width, groups, width, groups)]
    got = mp.mp3d_cache_read([t.cuda() for t in host], fmt, D, dt)
    for i in range(2):
        same(got[i], oracle.read(host[2 * i], host[2 * i + 1], fmt, D, dt))


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("fmt", FMT)
def test_rows_out_of_range_and_padding(fmt, dt):
    """Tokens past a sequence's count, or whose row is before or behind the
    cache, are dropped; reading such rows gives zeros."""
    B, T, H, D, rows = 6, 7, 2, 40, 10
    k, v = tk.randn((B, T, H, D), 3, dt), tk.randn((B, T, H, D), 4, dt)
    start = torch.tensor([0, -3, 6, 10, -100, 2 ** 31 - 1], dtype=torch.int32)
    count = torch.tensor([0, 7, 7, 3, 99, 5], dtype=torch.int32)
    cache = empty(B, rows, H, D, fmt)
    mp.mp3d_cache_write(k.cuda(), v.cuda(), cache, fmt, start=start.cuda(), count=count.cuda())
    check(k, v, fmt, cache, start, count)
    count[0] = -5
    got = mp.mp3d_cache_read(cache, fmt, D, dt, rows=T, start=start.cuda(), count=count.cuda())
    for i in range(2):
        held = oracle.read(cache[2 * i].cpu(), cache[2 * i + 1].cpu(), fmt, D, dt)
        want = torch.zeros((B, T, H, D), dtype=dt)
        for b in range(B):
            for t in range(min(T, int(count[b]))):
                if 0 <= int(start[b]) + t < rows:
                    want[b, t] = held[b, int(start[b]) + t]
        same(got[i], want)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
def test_groups_that_are_not_finite(dt, fmt):
    """A group with an infinity or a NaN is NaN, its neighbours are not."""
    k = tk.randn((1, 4, 2, 96), 5, dt)
    k[0, 0, 0, 40] = float("inf")
    k[0, 1, 1, 95] = float("-inf")
    k[0, 2, 0, 0] = float("nan")
    cache = empty(1, 4, 2, 96, fmt)
    mp.mp3d_cache_write(k.cuda(), k.cuda(), cache, fmt)
    check(k, k, fmt, cache, [0], None)
    got = mp.mp3d_cache_read(cache, fmt, 96, dt)[0].cpu()
    bad = torch.zeros((1, 4, 2, 3), dtype=torch.bool)
    bad[0, 0, 0, 1] = bad[0, 1, 1, 2] = bad[0, 2, 0, 0] = True
    assert torch.equal(torch.isnan(got), bad.repeat_interleave(32, -1))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("D", [64, 72])
def test_layouts(D, dt, fmt):
    """Inputs cut from a projection, caches token by token, and parts that
    start at any byte."""
    B, T, H, rows = 2, 33, 3, 50
    kv = tk.randn((B, T, 2 * H + 1, D + 1), 6, dt).cuda()
    start = torch.tensor([1, 17], dtype=torch.int32)
    width, groups = oracle.widths(fmt, D)
    for k, v in ((kv[:, :, :H, :D], kv[:, :, H:2 * H, 1:]),
                 (kv[:, :, :H, :D].contiguous(), kv[:, :, H:2 * H, :D].transpose(1, 2)
                  .contiguous().transpose(1, 2))):
        for extra in (0, 4, 3):
            cache = [torch.full((B, rows, H, n + extra), 0xA5, dtype=torch.uint8,
                                device="cuda")[..., extra:] for n in (width, groups, width, groups)]
            mp.mp3d_cache_write(k, v, cache, fmt, start=start.cuda())
            check(k.cpu(), v.cpu(), fmt, cache, start, None)
            got = mp.mp3d_cache_read(cache, fmt, D, dt, rows=T, start=start.cuda())
            for i in range(2):
                same(got[i], oracle.read(*oracle.write((k, v)[i].cpu(), fmt), fmt, D, dt))


def test_long_prompts():
    """More rows than one round of a workgroup takes, in every part the same
    as in a call by itself."""
    B, T, H, D = 3, 1531, 5, 72
    k, v = (tk.randn((B, T, H, D), n, torch.bfloat16).cuda() for n in (8, 9))
    for fmt in FMT:
        cache = empty(B, T, H, D, fmt)
        mp.mp3d_cache_write(k, v, cache, fmt)
        check(k.cpu(), v.cpu(), fmt, cache, [0] * B, None)
        got = mp.mp3d_cache_read(cache, fmt, D, torch.bfloat16)
        for t in (0, 700, T - 1):
            at = torch.full((B,), t, dtype=torch.int32, device="cuda")
            one = mp.mp3d_cache_read(cache, fmt, D, torch.bfloat16, rows=1, start=at)
            for a, b in zip(got, one):
                assert torch.equal(a[:, t:t + 1], b)


def test_rows_past_32_bits():
    """A cache whose rows are more than 2^32 bytes from its first."""
    rows, H, D = (1 << 25) + 5000, 1, 144
    cache = mp.mp3d_cache_empty(1, rows, H, D, "e4m3")
    for t in cache:
        t.zero_()
    k, v = (tk.randn((1, 9, H, D), n, torch.float16) for n in (10, 11))
    start = torch.tensor([rows - 9], dtype=torch.int32, device="cuda")
    mp.mp3d_cache_write(k.cuda(), v.cuda(), cache, "e4m3", start=start)
    got = mp.mp3d_cache_read(cache, "e4m3", D, torch.float16, rows=9, start=start)
    for i, x in enumerate((k, v)):
        same(got[i], oracle.read(*oracle.write(x, "e4m3"), "e4m3", D, torch.float16))
        assert int(cache[2 * i][:, :rows - 9].count_nonzero()) == 0


def test_nothing_to_do():
    for fmt in FMT:
        cache = empty(2, 4, 2, 32, fmt)
        e = torch.empty((2, 0, 2, 32), device="cuda")
        mp.mp3d_cache_write(e, e, cache, fmt)
        assert all(bool((t == 0xA5).all()) for t in cache)
        k, v = mp.mp3d_cache_read(cache, fmt, 32, torch.float32, rows=0)
        assert k.shape == v.shape == (2, 0, 2, 32)
        none = mp.mp3d_cache_empty(2, 0, 2, 32, fmt)
        x = torch.ones((2, 3, 2, 32), device="cuda")
        mp.mp3d_cache_write(x, x, none, fmt)
        k, v = mp.mp3d_cache_read(none, fmt, 32, torch.float32, rows=3)
        assert torch.equal(k, torch.zeros_like(x)) and torch.equal(v, torch.zeros_like(x))


def test_shapes_are_checked():
    x = torch.zeros((2, 3, 2, 40), device="cuda")
    c = empty(2, 8, 2, 40, "e4m3")
    for bad in ((c[0], c[1], c[2]), (c[0], c[2], c[1], c[3]), empty(2, 8, 2, 41, "e4m3"),
                empty(2, 8, 3, 40, "e4m3"), empty(1, 8, 2, 40, "e4m3"), empty(2, 8, 2, 40, "e2m1"),
                [t.float() for t in c], [t.cpu() for t in c],
                [t.transpose(2, 3).contiguous().transpose(2, 3) for t in c]):
        with pytest.raises(ValueError):
            mp.mp3d_cache_write(x, x, bad, "e4m3")
    n = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        mp.mp3d_cache_write(x, x, c, "e4m3", start=n)
    with pytest.raises(ValueError):
        mp.mp3d_cache_write(x, x, c, "e4m3", count=n.int()[:1])
    with pytest.raises(ValueError):
        mp.mp3d_cache_write(x, x[:, :2], c, "e4m3")
    with pytest.raises(TypeError):
        mp.mp3d_cache_write(x.double(), x.double(), c, "e4m3")
    with pytest.raises(TypeError):
        mp.mp3d_cache_read(c, "e4m3", 40, torch.float64)
    with pytest.raises(ValueError):
        mp.mp3d_cache_read(c, "e4m3", 41, torch.float32)


def test_capture_and_another_stream():
    """A write and a read captured once: each replay takes the rows and the
    tokens that are there then, with eager work between the replays."""
    B, T, H, D, fmt, dt = 3, 2, 2, 64, "e4m3", torch.bfloat16
    k, v = (torch.zeros((B, T, H, D), dtype=dt, device="cuda") for _ in range(2))
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache = empty(B, 16, H, D, fmt)

    def both():
        mp.mp3d_cache_write(k, v, cache, fmt, start=start)
        return mp.mp3d_cache_read(cache, fmt, D, dt)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in cache:
        t.zero_()
    want = [torch.zeros((B, 16, H, D), dtype=dt) for _ in range(2)]
    for n in range(4):
        new = [tk.randn((B, T, H, D), 20 + 2 * n + i, dt) for i in range(2)]
        k.copy_(new[0])
        v.copy_(new[1])
        start.copy_(torch.tensor([n, 14 - 3 * n, 2 * n], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for b in range(B):
                at = int(start[b])
                want[i][b, at:at + T] = oracle.read(*oracle.write(new[i][b], fmt), fmt, D, dt)
            same(got[i], want[i])
        mp.mp3d_cache_read(cache, fmt, D, dt)
