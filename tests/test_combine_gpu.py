"""moe_combine of more items than one launch has waves."""
import pytest
import torch

import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_combine_of_2_26_rows():
    """Rows of one 16-byte vector, so that every row is an item; the last waves take a second one."""
    T, N, S = (1 << 26) + 1003, 8, 5
    g = torch.Generator(DEV)
    g.manual_seed(1)
    Y = torch.randn((S, N), generator=g, device=DEV).bfloat16()
    slots = torch.randint(-1, S, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    weights = torch.randint(1, 4, (T, 1), generator=g, device=DEV, dtype=torch.int32).float()
    log(f"combine T={T} N={N}")
    out = gc.moe_combine(Y, slots, weights)
    # one product a row, rounded once: the same as torch's product in fp32
    table = (Y.float()[None] * torch.arange(4, device=DEV)[:, None, None]).bfloat16()
    table = torch.cat([table, torch.zeros((4, 1, N), dtype=torch.bfloat16, device=DEV)], dim=1)
    at = weights[:, 0].long() * (S + 1) + torch.where(slots[:, 0] < 0, S, slots[:, 0]).long()
    # (in parts: torch's own indexing of 2^26 rows and more gives zeros)
    for lo in range(0, T, 1 << 24):
        hi = min(T, lo + (1 << 24))
        assert torch.equal(out[lo:hi], table.reshape(-1, N)[at[lo:hi]]), lo
