"""CPU: the LDS that the kernel of shared tiles asks for, over everything its launch may be called with
(tests/host_plan/tile_lds.cpp includes the launch's own arithmetic)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_workgroups_fit_a_compute_unit(tmp_path):
    exe = str(tmp_path / "tile_lds")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", os.path.join(ROOT, "scale_gla_layer_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host_plan", "tile_lds.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert res.returncode == 0, res.stdout
