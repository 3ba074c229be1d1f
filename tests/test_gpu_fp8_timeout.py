"""Failure detection of the attention over the per-head e4m3 cache on tensor
memory and of the attention over whole prompts: their bounded waits run out
and the calls report it.

The build of the library that the failure-detection tests use
(KVQ_ATTN_STALL_TILE) makes the warps that issue the output products stop at
tile 2, as if their tensor work never completed, and shortens the role waits'
limit to about 10 ms.  Nothing hangs: the waits run out, every role leaves its
loop, products and copies in flight are drained, tensor memory is freed.

Checked, in a process of its own: KVQ_STATUS_TIMEOUT is set, rows whose
products never came are untouched, other rows are either untouched or right,
and the normal library then gives the same bits as before in the same process.
"""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
STALL_FLAGS = ["-DKVQ_ATTN_STALL_TILE=2", "-DKVQ_ATTN_WAIT_CYCLES=20000000LL"]


def test_waits_time_out_and_report():
    from fp8_quantized_paged_concat_gb300 import _build
    _build.build()
    library = _build.build(extra_flags=STALL_FLAGS, library=os.path.join(_build.PKG, "_lib", "libkvq_stall.so"),
                           objdir=os.path.join(_build.ROOT, "_build", "kvq_stall"))
    r = subprocess.run([sys.executable, os.path.join(HERE, "fp8_timeout_child.py"), library],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    reports = json.loads(r.stdout.strip().splitlines()[-1])
    assert [rep["call"] for rep in reports] == ["whole", "ranges", "gathered", "prompt 64", "prompt 128", "prompt 256"]
    for rep in reports:
        assert rep["status"] == 0x4, f"KVQ_STATUS_TIMEOUT alone: {rep}"
        assert rep["untouched"], f"a row whose products never came was written: {rep}"
        assert rep["others"], f"a row is neither untouched nor right: {rep}"
        assert rep["normal_status"] == 0 and rep["same"] and rep["finite"], rep
