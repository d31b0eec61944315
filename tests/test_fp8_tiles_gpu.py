"""gemm_fp8 through every kernel instance that its plan can choose, on operands
whose results are exact in any order of the sums."""
import pytest
import torch

import tensor_bf16_gemm_amd as gc
from fp8_cases import MANY_PEERS, exact_operands, instance, product
from gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", list(MANY_PEERS))
def test_every_place_of_the_peers_is_filled_again(rows):
    """15 peers, whose blocks pass through the waves' one or two places in LDS during the steps of K,
    each place read and filled again up to 120 times."""
    M, N, K = MANY_PEERS[rows]
    assert instance(gc.gemm_fp8_plan(M, N, K, 15), 15) == (rows, "peers")
    assert -(-K // 128) >= 15 * (rows // 32) + 2
    log(f"gemm_fp8 M={M} N={N} K={K} peers=15")
    ops = exact_operands(M, N, K, 15, rows)
    want = product(*ops)
    for _ in range(3):
        assert torch.equal(gc.gemm_fp8(*ops), want)
