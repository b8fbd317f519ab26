"""How attention over caches cuts its work, checked on the host (no GPU):
compiles tests/host/cached_plan_check.cpp with hipcc and runs it."""
import os
import subprocess

from bwd_max_pool3d_amd import _lib

HERE = os.path.dirname(os.path.abspath(__file__))


def test_long_caches_go_in_one_round_of_workgroups(tmp_path):
    """Codes of any alignment, and float32 over 64 channels, were cut for three
    workgroups a CU where two run at once."""
    where, name = os.path.split(os.path.abspath(_lib.load()._name))
    exe = tmp_path / "cached_plan_check"
    r = subprocess.run(["/opt/rocm/bin/hipcc", "-O2", "-std=c++17", "--offload-arch=gfx950",
                        os.path.join(HERE, "host", "cached_plan_check.cpp"), "-L" + where,
                        "-l:" + name, "-Wl,-rpath," + where, "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "cached plans: ok" in r.stdout
