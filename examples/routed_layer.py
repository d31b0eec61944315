"""One rank's share of a transformer layer with adapters and routed experts.

    python examples/routed_layer.py [--tokens 64] [--hidden 1024] [--experts 16] ...

The tokens of a batch, each of a request that may use an adapter of its own,
go through

    x -> projection summed over the tensor-parallel ranks (gemm_ar)
      -> + the requests' adapters                          (group_rows once a batch, lora_add)
      -> router: k experts per token, grouped              (moe_route)
      -> gate and up products of each expert's tokens      (grouped_gemm, silu_glu)
      -> down products                                     (grouped_gemm)
      -> weighted sum + the other ranks' partial sums      (moe_combine)

The projection is split along K over the ranks: x and the rows of its weights
are this rank's part, and so are the rows of the adapters' `down`.  Each rank
adds its own x . down . up to its own product, so the other ranks' partial
sums of the projection hold their adapters' parts too, and the sum of all is
the whole X . down . up.  The other ranks are buffers in this GPU's memory, as
everywhere in this package.  Prints the time of a pass and the busiest expert.
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_bf16_gemm_amd as gc  # noqa: E402


@dataclass
class Layer:
    """Weights of one rank: projection, adapters, router, experts."""
    proj: torch.Tensor        # [hidden, hidden]: this rank's rows of the projection
    down: torch.Tensor        # [adapters, hidden, rank]: the same rows of the adapters
    up: torch.Tensor          # [adapters, rank, hidden]
    scale: torch.Tensor       # [adapters]
    router: torch.Tensor      # [hidden, experts]
    w1: torch.Tensor          # [experts, hidden, 2 * inner]: gate and up columns
    w2: torch.Tensor          # [experts, inner, hidden]


def make_layer(hidden: int, inner: int, experts: int, adapters: int, rank: int, seed: int = 0) -> Layer:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def w(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * shape[-2] ** -0.5

    return Layer(w(hidden, hidden), w(adapters, hidden, rank), w(adapters, rank, hidden),
                 torch.rand(adapters, generator=g, device="cuda") + 0.5, w(hidden, experts),
                 w(experts, hidden, 2 * inner), w(experts, inner, hidden))


def forward(p: Layer, x, adapters, proj_peers, moe_peers, k: int, ranks: int):
    """Tokens x [T, hidden]; adapters: gc.group_rows of the tokens' adapters (-1: none); proj_peers
    and moe_peers [ranks - 1, T, hidden]: the other ranks' partial sums (of the projection: with their
    adapters' parts).  Returns the layer's output and the routing."""
    h = gc.gemm_ar(x, p.proj, proj_peers, R=ranks, rank=0)
    gc.lora_add(h, x, p.down, p.up, p.scale, adapters.offsets, adapters.rows, out=h)
    r = gc.moe_route((h @ p.router).float(), k)
    a = gc.grouped_gemm(h, p.w1, r.offsets, r.rows, act="silu_glu")
    y = gc.grouped_gemm(a, p.w2, r.offsets)
    return gc.moe_combine(y, r.slots, r.weights, moe_peers), r


def make_batch(tokens: int, hidden: int, adapters: int, ranks: int, seed: int = 1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    ids = torch.randint(-1, adapters, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    return r(tokens, hidden), ids, r(ranks - 1, tokens, hidden), r(ranks - 1, tokens, hidden)


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, v in dict(tokens=64, hidden=1024, inner=512, experts=16, k=4, adapters=8, rank=16, ranks=8,
                        steps=50).items():
        a.add_argument(f"--{name}", type=int, default=v)
    a = a.parse_args()
    p = make_layer(a.hidden, a.inner, a.experts, a.adapters, a.rank)
    x, ids, proj_peers, moe_peers = make_batch(a.tokens, a.hidden, a.adapters, a.ranks)
    groups = gc.group_rows(ids, a.adapters)           # once a batch: every layer uses it
    for _ in range(3):
        out, routing = forward(p, x, groups, proj_peers, moe_peers, a.k, a.ranks)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        out, routing = forward(p, x, groups, proj_peers, moe_peers, a.k, a.ranks)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / a.steps * 1e6
    busiest = int((routing.offsets[1:] - routing.offsets[:-1]).max())
    print(f"{a.tokens} tokens, {a.experts} experts, {a.adapters} adapters: {us:.1f} us a layer, busiest expert "
          f"{busiest} rows, output finite: {bool(torch.isfinite(out).all())}")


if __name__ == "__main__":
    main()
