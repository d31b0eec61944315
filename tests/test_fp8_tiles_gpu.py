"""gemm_fp8 through every kernel instance that its plan can choose, on operands
whose results are exact in any order of the sums."""
import math

import pytest
import torch

import tensor_bf16_gemm_amd as gc
from fp8_cases import E4M3, MANY_PEERS, NO_K, STREAMS, TILES, exact_operands, instance, product
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
SENTINEL = 0x7FC1


def filled(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)


def laid_out(sa, form):
    """(scales of that layout, the same values contiguous); what lies between them is NaN."""
    M, kb = sa.shape
    if form == "contiguous":
        s = sa
    elif form == "columns first":
        s = sa.t().contiguous().t()
    elif form == "odd rows":
        s = torch.full((M, kb + 3 - kb % 2), math.nan, device=DEV)[:, 1:kb + 1]
        s.copy_(sa)
    elif form == "every fourth":
        s = torch.full((M, 4 * kb), math.nan, device=DEV)[:, ::4]
        s.copy_(sa)
    elif form == "one row":
        s = sa[:1].expand(M, -1)
    else:
        s = sa[:, :1].expand(-1, kb)
    return s, s.contiguous()


@pytest.mark.parametrize("form", ["contiguous", "columns first", "odd rows", "every fourth", "one row", "one block"])
@pytest.mark.parametrize("which", list(TILES), ids=lambda w: f"{w[0]} {w[1]}")
def test_scales_of_any_strides(which, form):
    """Exact results whatever the scales' strides, and nothing written around the output."""
    M, N, K, peers = TILES[which]
    assert instance(gc.gemm_fp8_plan(M, N, K, peers), peers) == which
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers} {which} scales {form}")
    A, sa, B, sb, p = exact_operands(M, N, K, peers, M + K)
    s, values = laid_out(sa, form)
    buf = filled(M + 3, N)
    got = gc.gemm_fp8(A, s, B, sb, p, out=buf[1:M + 1])
    assert torch.equal(got, product(A, values, B, sb, p))
    keep = buf.view(torch.int16)
    assert (keep[0] == SENTINEL).all() and (keep[M + 1:] == SENTINEL).all()


@pytest.mark.parametrize("which", list(TILES), ids=lambda w: f"{w[0]} {w[1]}")
def test_not_finite_stays_in_its_row_or_column(which):
    M, N, K, peers = TILES[which]
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers} {which} with infinities and NaN")
    A, sa, B, sb, p = exact_operands(M, N, K, peers, M + N)
    want = product(A, sa, B, sb, p)
    a, b, s = A.clone(), B.clone(), sa.clone()
    a.view(torch.uint8)[M - 1, K - 1] = 0x7F              # NaN in the last row's last block
    s[1, 0] = math.inf
    got = gc.gemm_fp8(a, s, B, sb, p)
    assert torch.isnan(got[M - 1]).all() and not torch.isfinite(got[1]).any()
    rest = torch.ones(M, dtype=torch.bool, device=DEV)
    rest[[1, M - 1]] = False
    assert torch.equal(got[rest], want[rest])
    b.view(torch.uint8)[17, K - 1] = b.view(torch.uint8)[N - 1, 0] = 0xFF
    got = gc.gemm_fp8(A, sa, b, sb, p)
    rest = torch.ones(N, dtype=torch.bool, device=DEV)
    rest[[17, N - 1]] = False
    assert torch.isnan(got[:, [17, N - 1]]).all() and torch.equal(got[:, rest], want[:, rest])
    if peers:
        q = p.clone()
        q[peers - 1, M - 1, N - 1], q[0, 0, 0] = math.nan, -math.inf
        got = gc.gemm_fp8(A, sa, B, sb, q)
        assert torch.isnan(got[M - 1, N - 1]) and got[0, 0] == -math.inf
        got[M - 1, N - 1], got[0, 0] = want[M - 1, N - 1], want[0, 0]
        assert torch.equal(got, want)


@pytest.mark.parametrize("rows", list(NO_K))
def test_no_k(rows):
    """K = 0 through the tiles: the peers' sum."""
    M, N = NO_K[rows]
    assert instance(gc.gemm_fp8_plan(M, N, 0, 5), 5) == (rows, "peers")
    log(f"gemm_fp8 M={M} N={N} K=0")
    p = exact_operands(M, N, 0, 5, rows)[4]
    none = lambda n: torch.empty((n, 0), dtype=E4M3, device=DEV)  # noqa: E731
    got = gc.gemm_fp8(none(M), torch.empty((M, 0), device=DEV), none(N), torch.empty((-(-N // 128), 0), device=DEV), p)
    assert torch.equal(got, p.float().sum(0).bfloat16())


@pytest.mark.parametrize("peers", [0, 2])
@pytest.mark.parametrize("which", list(STREAMS), ids=lambda w: f"{w[0]}x{w[1]}")
def test_streams_past_one_load_of_scales(which, peers):
    """K beyond the 64 blocks whose scales the streaming kernel holds at a time."""
    M, N, K = STREAMS[which]
    assert instance(gc.gemm_fp8_plan(M, N, K, peers), peers) == which
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers} {which}")
    for seed in range(3):
        A, sa, B, sb, p = exact_operands(M, N, K, peers, seed)
        want = product(A, sa, B, sb, p)
        assert torch.equal(gc.gemm_fp8(A, sa, B, sb, p), want)
        assert torch.equal(gc.gemm_fp8(A, laid_out(sa, "columns first")[0], B, sb, p), want)


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
