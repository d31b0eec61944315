"""What can be checked of gemm_fp8's kernels without a GPU."""
import os
import re

import tensor_bf16_gemm_amd as gc
from fp8_cases import MANY_PEERS, NO_K, STREAMS, TILES, instance

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_places_of_the_peers_are_read_before_they_are_filled_again():
    """A wave's place in LDS for a block of a peer is filled by a load that the compiler does not
    track, so the wait for what was read from it stands in the source, right before the load.  (No
    result shows its absence while the compiler happens to wait there by itself.)"""
    text = open(os.path.join(ROOT, "tensor_bf16_gemm_amd", "csrc", "fp8_gemm.hpp")).read()
    text = re.sub(r"//[^\n]*", "", text)
    asked = [m.start() for m in re.finditer(r"\bask\(part", text)]
    assert asked
    for at in asked:
        assert text[:at].rstrip().endswith("wait_lgkmcnt0();")


def test_the_cases_reach_every_instance():
    """Every kernel that the host side can launch is run by the sizes of fp8_cases."""
    plan = gc.gemm_fp8_plan
    assert {(r, e) for r in (64, 128, 224, 256) for e in ("plain", "peers", "cut")} == set(TILES)
    for want, (M, N, K, peers) in TILES.items():
        assert instance(plan(M, N, K, peers), peers) == want
    assert {(16, 16), (16, 32), (32, 16), (32, 32), (32, 64), (64, 32)} == set(STREAMS)
    for want, (M, N, K) in STREAMS.items():
        assert K > 8192 and K % 128 != 0
        for peers in (0, 2):
            assert instance(plan(M, N, K, peers), peers) == want
    for rows, (M, N, K) in MANY_PEERS.items():
        assert instance(plan(M, N, K, 15), 15) == (rows, "peers")
    for rows, (M, N) in NO_K.items():
        assert instance(plan(M, N, 0, 5), 5) == (rows, "peers")
