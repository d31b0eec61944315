"""Ranks: experts spread over them, where each groups the pairs of its own and the
others' results come in as partial sums; adapters beside a split projection."""
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


@pytest.mark.parametrize("T", [1, 50])
def test_adapters_of_a_projection_split_along_k(T):
    """Each rank holds a slice of K of the rows, the projection and the adapters' down; the partial sums
    that the others publish hold their adapters' parts.  Every rank ends with the whole projection and the
    whole adapters' sum."""
    ranks, Kr, N, r, G = 4, 64, 136, 16, 3
    g = torch.Generator()
    g.manual_seed(T)
    X = torch.randn((ranks, T, Kr), generator=g).bfloat16()
    W = (torch.randn((ranks, Kr, N), generator=g) * (ranks * Kr) ** -0.5).bfloat16()
    down = (torch.randn((ranks, G, Kr, r), generator=g) * (ranks * Kr) ** -0.5).bfloat16()
    up = (torch.randn((G, r, N), generator=g) * r ** -0.5).bfloat16()
    scale = torch.rand(G, generator=g) + 0.5
    ids = torch.randint(-1, G, (T,), generator=g, dtype=torch.int32)
    grp = gc.group_rows(ids.to(DEV), G)
    want, mag = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
    parts = []
    for q in range(ranks):
        base = X[q].double() @ W[q].double()
        own, _ = ref.lora(base, X[q], down[q], up, scale, ids)
        want, mag = want + own, mag + own.abs()
        parts.append(own.bfloat16())                    # as rank q publishes it
    log(f"split projection T={T}")
    for q in range(ranks):
        peers = torch.stack([p for i, p in enumerate(parts) if i != q]).to(DEV)
        x = X[q].to(DEV)
        h = gc.gemm_ar(x, W[q].to(DEV), peers, R=ranks, rank=q)
        first = h.double().cpu()
        gc.lora_add(h, x, down[q].to(DEV), up.to(DEV), scale.to(DEV), grp.offsets, grp.rows, out=h)
        # each partial is rounded once, the projection's output and the adapters' once each; all sums
        # together (512 terms at most) are off by far less than one more such rounding
        bound = ref.BF * (mag + first.abs() + want.abs()) * 1.05 + 2.0 ** -12 * mag
        assert torch.all((h.double().cpu() - want).abs() <= bound)
