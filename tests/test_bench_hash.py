"""bench.py's stored traffic counters go with everything that decides which
pooling kernel runs and how it was compiled."""
import os
import re

import bench
from bwd_max_pool3d_amd import _build

TOKENS = {"api_tokens.hip", "rope.hip", "gated_norm.hip", "attention_fwd.hip",
          "attention_split.hip", "attention_bwd.hip", "attention_order.hip"}


def test_every_pooling_source_and_what_it_includes():
    assert set(_build.SOURCES) - TOKENS <= set(_build.POOL_KERNELS)
    for name in _build.POOL_KERNELS:
        with open(os.path.join(_build.CSRC, name)) as f:
            used = re.findall(r'#include "([^"/]+)"', f.read())
        assert set(used) <= set(_build.POOL_KERNELS), name


def test_sources_and_flags_change_the_hash(monkeypatch, tmp_path):
    before = bench.kernel_source_hash()
    monkeypatch.setattr(_build, "HIPCC_FLAGS", _build.HIPCC_FLAGS + ["-g"])
    assert bench.kernel_source_hash() != before
    monkeypatch.undo()
    for name in _build.POOL_KERNELS:
        with open(os.path.join(_build.CSRC, name)) as f:
            (tmp_path / name).write_text(f.read())
    monkeypatch.setattr(_build, "CSRC", str(tmp_path))
    assert bench.kernel_source_hash() == before
    (tmp_path / "api.hip").write_text("// another dispatch\n")
    assert bench.kernel_source_hash() != before
