"""Failure detection of the per-head attention on tensor memory (calls of more
than 32 query rows per request and key head): its bounded waits run out and
the call reports it.

A build of the library used only by the failure-detection tests
(KVQ_ATTN_STALL_TILE) makes the warp that issues the output products stop at
tile 2, as if its tensor work never completed, and shortens the role waits'
limit (KVQ_ATTN_WAIT_CYCLES, about 10 ms).  Nothing hangs: the waits that
nothing will satisfy run out, every role leaves its loop, the two issuing
warps drain the products they issued, the kernel frees its tensor memory and
returns; a second launch that joins key ranges skips the rows of a range that
gave up.

Checked, in a process of its own: KVQ_STATUS_TIMEOUT is set, out and lse are
untouched, whole and in ranges, and the normal library then gives the same
bits as before on the same device in the same process.
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
    r = subprocess.run([sys.executable, os.path.join(HERE, "per_head_timeout_child.py"), library],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    reports = json.loads(r.stdout.strip().splitlines()[-1])
    assert [rep["splits"] for rep in reports] == [1, 2]
    for rep in reports:
        assert rep["status"] == 0x4, f"KVQ_STATUS_TIMEOUT alone: {rep}"
        assert rep["untouched"], f"a row whose products never came was written: {rep}"
        assert rep["normal_status"] == 0 and rep["same"] and rep["finite"], rep
