"""lora_add where its middle activations are at the edges of their types."""
import math

import pytest
import torch

import grouped_ref as ref
import tensor_bf16_gemm_amd as gc
from adapter_cases import COLUMNS, ROWS
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = math.inf


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def run(base, X, down, up, scale, ids, out=None):
    off, rows, _ = gc.group_rows(ids.to(DEV), down.shape[0])
    d = [t.to(DEV) for t in (base, X, down, up, scale)]
    return gc.lora_add(*d, off, rows, out=d[0] if out == "base" else out)


def pieces(a):
    """The bits 23..16, 15..8 and 7..0 of whole numbers below 2^24: each exact in bf16."""
    return a & 0xFF0000, a & 0xFF00, a & 0xFF


# (rows, adapters): few rows per adapter, and many
@pytest.mark.parametrize("M,G", [(1, 1), (40, 5), (150, 2), (70, 1)])
@pytest.mark.parametrize("r", [8, 16, 40, 72, 104, 128])
def test_middle_sums_keep_all_bits(M, G, r):
    """H holds pairs of a 24-bit number and the same with its low byte cleared, which up subtracts:
    the low bytes are left, exactly.  Every fp32 sum on the way is a whole number below 2^24 times
    a power of two, so the only rounding is that of the output."""
    g = gen(M + r)
    N, pairs = 136, r // 2
    K = (3 * pairs + 7) // 8 * 8
    a = torch.randint(1 << 23, 1 << 24, (M, pairs), generator=g)
    X, down = torch.zeros(M, K), torch.zeros(G, K, r)
    for p in range(pairs):
        for i, part in enumerate(pieces(a[:, p])):
            X[:, 3 * p + i] = part.float()
            down[:, 3 * p + i, 2 * p] = 1.0
            if i < 2:
                down[:, 3 * p + i, 2 * p + 1] = 1.0
    up = torch.zeros(G, r, N)
    up[:, 0::2], up[:, 1::2] = 1.0, -1.0
    up[:, :, 1::3] *= 0.5
    scale = torch.tensor([2.0 ** -(i % 3) for i in range(G)])
    ids = torch.randint(0, G, (M,), generator=g, dtype=torch.int32)
    log(f"whole middle sums M={M} G={G} r={r}")
    got = run(torch.zeros(M, N).bfloat16(), X.bfloat16(), down.bfloat16(), up.bfloat16(), scale, ids)
    low = (a & 0xFF).sum(1).double()
    want = (low * scale[ids.long()].double())[:, None] * up[0, 0].double()
    assert torch.equal(got.cpu(), want.bfloat16())


@pytest.mark.parametrize("M,G", [(12, 2), (90, 2)])
@pytest.mark.parametrize("r", [8, 64, 96])
def test_infinite_and_largest_middle_sums(M, G, r):
    """An infinite H, one that lies above the largest bf16, and infinite and NaN weights give what
    the sum in 64 bits gives, in their own rows and columns only."""
    g = gen(M * r)
    K, N = 72, 200
    X, base = randn(g, M, K), randn(g, M, N)
    down, up = randn(g, G, K, r, scale=K ** -0.5), randn(g, G, r, N, scale=r ** -0.5)
    X[:, :8] = 0.0
    down[:, :8] = 0.0
    down[:, 3] = 1.0                                    # X[.., 3] reaches every middle value
    down[:, 5:8, 0] = 1.0                               # X[.., 5:8] the first one alone
    down[:, 5:8, 1:] = 0.0
    up[:, :, :100] = up[:, :, :100].abs() + 2.0 ** -10  # an infinite H gives inf here, NaN among the others
    ids = torch.arange(M, dtype=torch.int32) % G
    X[2, 3], X[5, 3], X[M - 1, 3] = INF, -INF, math.nan
    # 2^128 - 2^118: finite, and nearer to 2^128 than to the largest bf16; the adapter's products
    # with it stay finite (the rest of the row is zero)
    big = torch.tensor([2.0 ** 128 - 2.0 ** 120, 2.0 ** 119, 2.0 ** 118], dtype=torch.float64).bfloat16()
    X[6] = 0.0
    X[6, 5:8] = big
    up[:, 0] = up[:, 0].abs().clamp(0.01, 0.5)
    up[1, 1, 150], up[1, 2, 151], up[1, 3, 152] = INF, -INF, math.nan
    scale = torch.tensor([1.0, 0.5])
    want, tol = ref.lora(base, X, down, up, scale, ids)
    log(f"infinite middle sums M={M} r={r}")
    for out in (None, "base"):
        got = run(base, X, down, up, scale, ids, out).cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        odd = torch.isinf(want)
        assert torch.equal(got[odd], want[odd])
        ok = torch.isfinite(want)
        # fp32 sums of an adapter with an infinite weight have no bound; their finite ones do
        assert torch.all((got - want).abs()[ok] <= tol[ok])
    assert odd[2, :100].all() and odd[5, :100].all() and ok[6].all()


@pytest.mark.parametrize("M,G", [(24, 2), (150, 2)])
def test_rows_of_no_adapter_are_base_bit_by_bit(M, G):
    """Every bf16 there is, zeros with a sign and NaN with a payload among them."""
    g = gen(M)
    N = (1 << 16) // M // 8 * 8 + 8
    bits = torch.arange(M * N, dtype=torch.int32) % (1 << 16) - (1 << 15)
    base = bits.to(torch.int16).view(torch.bfloat16).reshape(M, N)
    ids = torch.full((M,), -1, dtype=torch.int32)
    ids[M // 2] = 1
    got = run(base, randn(g, M, 40), randn(g, G, 40, 16), randn(g, G, 16, N), torch.ones(G), ids).cpu()
    free = ids < 0
    assert torch.equal(got[free].view(torch.int16), base[free].view(torch.int16))


@pytest.mark.parametrize("M,K,N,r,sizes", [c[:5] for c in ROWS + COLUMNS],
                         ids=lambda v: f"{len(v)}groups" if isinstance(v, list) else str(v))
def test_walks_of_several_blocks(M, K, N, r, sizes):
    """Against the 64-bit form, elementwise; apart from base and in its place."""
    g, G = gen(M + N + r), len(sizes)
    dg = torch.Generator(DEV)
    dg.manual_seed(M + N)
    ids = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in enumerate(sizes)]
                    + [torch.full((M - sum(sizes),), -1, dtype=torch.int32)])
    ids = ids[torch.randperm(M, generator=g)]
    X, down = randn(g, M, K).to(DEV), randn(g, G, K, r, scale=K ** -0.5).to(DEV)
    up = randn(g, G, r, N, scale=r ** -0.5).to(DEV)
    base = torch.randn((M, N), generator=dg, device=DEV).bfloat16()
    scale = torch.randn(G, generator=g).to(DEV)
    log(f"lora M={M} K={K} N={N} r={r} G={G}")
    want, tol = ref.lora(base, X, down, up, scale, ids.to(DEV))
    off, rows, _ = gc.group_rows(ids.to(DEV), G)
    got = gc.lora_add(base, X, down, up, scale, off, rows)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[0].tolist())
    same = gc.lora_add(base, X, down, up, scale, off, rows, out=base)
    assert same is base and torch.equal(same, got)
