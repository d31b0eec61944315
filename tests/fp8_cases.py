"""Sizes of gemm_fp8 that reach every kernel instance, and operands whose products are exact."""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn

# (tile rows, end) -> (M, N, K, peers): the tiles through LDS, none of whose sizes is a multiple of
# the tile's.
TILES = {
    (64, "plain"): (500, 4104, 656, 0), (64, "peers"): (500, 4104, 656, 3), (64, "cut"): (115, 4280, 7168, 0),
    (128, "plain"): (1800, 2056, 1424, 0), (128, "peers"): (1800, 2056, 1424, 3), (128, "cut"): (500, 4104, 4112, 1),
    (224, "plain"): (2000, 4104, 400, 0), (224, "peers"): (2000, 4104, 400, 3), (224, "cut"): (2146, 1976, 4112, 1),
    (256, "plain"): (2040, 6664, 656, 0), (256, "peers"): (2040, 6664, 656, 3), (256, "cut"): (689, 6016, 6144, 1)}

# (tile rows, tile columns) -> (M, N, K): streaming, past the 64 blocks of K whose scales are loaded
# at a time, with a last chunk and a last block that are not whole.
STREAMS = {(16, 16): (5, 72, 16400), (16, 32): (1, 4408, 8336), (32, 16): (2188, 40, 8336),
           (32, 32): (18, 4384, 8208), (32, 64): (33, 4192, 8336), (64, 32): (2845, 136, 8336)}

# tile rows -> (M, N, K): 15 peers, all of whose blocks enter during the steps of K.
MANY_PEERS = {64: (517, 4896, 4048), 128: (526, 7304, 8064), 224: (2692, 2856, 13824), 256: (1801, 7248, 15568)}

# tile rows -> (M, N): K 0 and peers.
NO_K = {64: (161, 8224), 128: (4097, 784), 224: (4654, 1544), 256: (1572, 8200)}


def instance(plan, peers):
    """(tile rows, end) of a plan of tiles through LDS, (tile rows, tile columns) of a streaming one."""
    if plan["tile_cols"] < 256:
        return plan["tile_rows"], plan["tile_cols"]
    return plan["tile_rows"], "cut" if plan["splits"] > 1 else "peers" if peers else "plain"


def exact_operands(M, N, K, peers, seed, device="cuda"):
    """(A, a_scales, B, b_scales, partials) of whole numbers up to 2, scales of 1/2, 1 and 2 and peers
    up to 64: every product with its scales is a multiple of 1/4, and sums of fewer than 2^17
    products are exact in fp32, in any order (and the products of 8 neighbouring k, 1 to 4, lose
    nothing inside a matrix instruction)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device=device).float()  # noqa: E731
    kb = -(-K // 128)
    return (ints(-2, 2, M, K).to(E4M3), torch.exp2(ints(-1, 1, M, kb)), ints(-2, 2, N, K).to(E4M3),
            torch.exp2(ints(-1, 1, -(-N // 128), kb)), ints(-64, 64, peers, M, N).bfloat16() if peers else None)


def product(A, sa, B, sb, p):
    """gemm_fp8 of finite operands in 64 bits, rounded to bf16 once (by way of fp32, which holds these
    sums exactly)."""
    M, K = A.shape
    a = A.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    b = B.double() * sb.double().repeat_interleave(128, 0)[:B.shape[0]].repeat_interleave(128, 1)[:, :K]
    out = a @ b.t()
    if p is not None:
        out += p.double().sum(0)
    assert torch.equal(out.float().double(), out)
    return out.bfloat16()
