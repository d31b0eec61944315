"""Calls of the routed and grouped operators at the edges of what they take
(no GPU needed).  A call that might end the process runs in one of its own."""
import os
import subprocess
import sys

import pytest

import tensor_bf16_gemm_amd as gc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def in_a_process(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    return r.stdout.strip()


@pytest.mark.parametrize("T,k", [(1, 8192), (3, 8192), (2, 100_000), (1, 1 << 24)])
def test_group_rows_of_wide_rows(T, k):
    """Rows longer than any block of items: without the workspace these are refused, not divided by 0."""
    code = ("import tensor_bf16_gemm_amd as gc; P = 0x7F0000000000; "
            f"print(gc.lib().gemm_coll_group_rows(P, {T}, {k}, 8, P, P, P, None, 0, None))")
    assert in_a_process(code) == str(gc.GC_EINVAL)
