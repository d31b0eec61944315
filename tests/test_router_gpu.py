"""moe_route and group_rows at block sizes and row lengths of their own, each
against its plain 64-bit form."""
import pytest
import torch

import grouped_ref as ref
import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("T,k,groups", [(3, 17, 5), (1, 1025, 9), (2, 8191, 7), (1, 8192, 8), (3, 8193, 300),
                                        (1, 100_000, 1024), (0, 9000, 4)])
def test_group_rows_of_wide_rows(T, k, groups):
    ids = torch.randint(-1, groups + 1, (T, k), generator=gen(k), dtype=torch.int32)
    log(f"group_rows T={T} k={k} groups={groups}")
    for got, want, name in zip(gc.group_rows(ids.to(DEV), groups), ref.group(ids, groups),
                               ("offsets", "rows", "slots")):
        assert torch.equal(got.cpu(), want), name
