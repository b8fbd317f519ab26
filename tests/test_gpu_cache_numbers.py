"""Every code under every scale, read in every type, and every 16-bit number
written under every scale at which it has a code that is not 0."""
import pytest
import torch

import _caches as oracle
import _tokens as tk
import bwd_max_pool3d_amd as mp
from test_gpu_cache import same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", tk.TYPES, ids=tk.name_of)
@pytest.mark.parametrize("fmt", oracle.FORMATS)
@pytest.mark.parametrize("cut", [0, 1])
def test_all_codes_under_all_scales(cut, fmt, dt):
    """Row s: all codes, all groups under the scale byte s.  cut: a channel
    fewer, which goes byte by byte."""
    D = 256 - cut                                          # e2m1: the sixteen codes, 16 times
    width, groups = oracle.widths(fmt, D)
    row = torch.arange(width) if fmt == "e4m3" else torch.arange(width) * 2 % 16 * 17 + 16
    codes = (row % 256).to(torch.uint8).expand(1, 256, 1, width).contiguous()
    scales = torch.arange(256).to(torch.uint8)[None, :, None, None].expand(1, 256, 1, groups)
    cache = [t.contiguous().cuda() for t in (codes, scales, codes, scales)]
    want = oracle.read(codes, scales, fmt, D, dt)
    for got in mp.mp3d_cache_read(cache, fmt, D, dt):
        same(got, want)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=tk.name_of)
@pytest.mark.parametrize("fmt", oracle.FORMATS)
def test_all_numbers_of_16_bits(fmt, dt):
    """Groups of 31 numbers that follow each other and one 2^n times the largest
    of them, n up to where their codes are 0."""
    bits = torch.arange(1 << 16).to(torch.int32)
    bits = torch.cat((bits, bits[:(-len(bits)) % 31])).view(-1, 31)
    x = bits.to(torch.int16).view(dt)                      # (groups, 31)
    largest = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().double().amax(1)
    rows = []
    for n in range(20 if fmt == "e4m3" else 6):
        top = (largest * 2.0 ** n).clamp(max=oracle.LARGEST[dt]).to(dt)
        rows.append(torch.cat((x, top[:, None]), 1))
    x = torch.cat(rows)[None, :, None]                     # (1, T, 1, 32)
    codes, scales = oracle.write(x, fmt)
    cache = mp.mp3d_cache_empty(1, x.shape[1], 1, 32, fmt)
    mp.mp3d_cache_write(x.cuda(), x.cuda(), cache, fmt)
    for i in range(2):
        same(cache[2 * i], codes, "codes")
        same(cache[2 * i + 1], scales, "scales")
