"""The cache attention's work list, checked on the host (no GPU): tests/attn_check.cu."""
import os
import subprocess

import pytest

from gated_pooling_gb300 import build as gb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_shares_fit_the_largest_calls(tmp_path):
    try:
        cc = gb.nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    exe = str(tmp_path / "attn_check")
    res = subprocess.run(
        [cc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr", "-I",
         os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "gated_pooling_gb300", "csrc"),
         os.path.join(ROOT, "tests", "attn_check.cu"), "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.startswith("ok "), run.stdout + run.stderr
