"""The per-head attention's choice of key ranges and row block, which is host
arithmetic (tests/c/per_head_plan_check.cpp); about a second."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_default_ranges_are_sized_for_the_block_that_runs(tmp_path):
    exe = tmp_path / "per_head_plan_check"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I" + os.path.join(ROOT, "include"),
                           "-I" + os.path.join(ROOT, "fp8_quantized_paged_concat_gb300", "csrc"),
                           os.path.join(HERE, "c", "per_head_plan_check.cpp"), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert "other block 0, out of limits 0" in r.stdout and "split 0" not in r.stdout
