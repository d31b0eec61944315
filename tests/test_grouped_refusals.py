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


@pytest.mark.parametrize("T,E,k", [(129, 64, 8), (1025, 64, 1), (342, 300, 3), (65, 8, 16)])
def test_more_than_1024_pairs_need_the_workspace(T, E, k):
    P = 0x7F0000000000
    L = gc.lib()
    assert L.gemm_coll_moe_route(P, 0, E, T, E, k, 0, None, 1, 1.0, P, P, P, P, P, None, 0, None) == gc.GC_EINVAL
    assert L.gemm_coll_group_rows(P, T, k, E, P, P, P, None, 0, None) == gc.GC_EINVAL
