"""What can be checked of gemm_fp8's kernels without a GPU."""
import os
import re

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
