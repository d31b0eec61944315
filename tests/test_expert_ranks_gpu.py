"""Experts spread over ranks: each groups the pairs of its own experts, and the
other ranks' results come in as partial sums."""
import pytest
import torch

import grouped_ref as ref
import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,ranks", [(1, 4), (37, 2), (300, 4)])
def test_experts_of_several_ranks(T, ranks):
    local, k, K, F = 3, 4, 72, 40
    E = local * ranks
    g = torch.Generator()
    g.manual_seed(T)
    x = torch.randn((T, K), generator=g).bfloat16().to(DEV)
    W1 = (torch.randn((E, K, 2 * F), generator=g) * K ** -0.5).bfloat16().to(DEV)
    W2 = (torch.randn((E, F, K), generator=g) * F ** -0.5).bfloat16().to(DEV)
    logits = torch.randn((T, E), generator=g)
    logits[T // 2] = -torch.inf                        # a token of no expert
    r = gc.moe_route(logits.to(DEV), k)
    log(f"T={T} ranks={ranks}")
    mine = []
    for first in range(0, E, local):
        s = gc.group_rows(r.ids - first, local)
        S = T * k
        h = torch.full((S, F), torch.nan, dtype=torch.bfloat16, device=DEV)    # rows of other ranks stay NaN
        y = torch.full((S, K), torch.nan, dtype=torch.bfloat16, device=DEV)
        gc.grouped_gemm(x, W1[first:first + local], s.offsets, s.rows, out=h, act="silu_glu")
        gc.grouped_gemm(h, W2[first:first + local], s.offsets, out=y)
        part = gc.moe_combine(y, s.slots, r.weights)
        ref.check(part, *ref.combine(y.cpu(), s.slots.cpu(), r.weights.cpu()), f"experts from {first}")
        mine.append((y, s.slots, part))
    for q, (y, slots, _) in enumerate(mine):
        others = torch.stack([m[2] for p, m in enumerate(mine) if p != q])
        out = gc.moe_combine(y, slots, r.weights, others)
        ref.check(out, *ref.combine(y.cpu(), slots.cpu(), r.weights.cpu(), others.cpu()), f"rank {q}")
    # every pair is on one rank
    there = sum((s >= 0).int() for _, s, _ in mine)
    assert torch.equal(there, (r.ids >= 0).int())
