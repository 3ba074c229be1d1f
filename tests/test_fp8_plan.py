"""The choice of key ranges, row block and gather of the attention over the
e4m3 cache, which is host arithmetic (tests/c/fp8_plan_check.cpp); about a
second."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_defaults_fit_the_calls_they_are_for(tmp_path):
    exe = tmp_path / "fp8_plan_check"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I" + os.path.join(ROOT, "include"),
                           "-I" + os.path.join(ROOT, "fp8_quantized_paged_concat_gb300", "csrc"),
                           os.path.join(HERE, "c", "fp8_plan_check.cpp"), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert "other block 0, out of limits 0, no room 0" in r.stdout and "gathers 0" not in r.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_defaults_that_gather_fit_their_room_and_fill_the_gpu(tmp_path):
    exe = tmp_path / "fp8_gather_check"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I" + os.path.join(ROOT, "include"),
                           "-I" + os.path.join(ROOT, "fp8_quantized_paged_concat_gb300", "csrc"),
                           os.path.join(HERE, "c", "fp8_gather_check.cpp"), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
