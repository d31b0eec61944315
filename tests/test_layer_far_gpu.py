"""Operands just below 2 GiB, and peers' blocks further apart than 32 bits
count bytes, on values whose sums are exact (gemm_fp8) or against the same
peers close together."""
import pytest
import torch

import tensor_bf16_gemm_amd as gc
from fp8_cases import exact_operands, instance, product
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
FAR = (1 << 31) + 8                                      # elements from a peer to the next: 2^32 bytes and 16


@pytest.mark.parametrize("peers", [0, 2])
def test_rows_to_two_gibibytes(peers):
    M, N, K = 262_143, 264, 8192                         # A: 2^31 - 8192 bytes
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers}")
    A, sa, B, sb, p = exact_operands(M, N, K, peers, 1)
    got = gc.gemm_fp8(A, sa, B, sb, p)
    for at in (slice(0, 300), slice(131_000, 131_300), slice(M - 300, M)):
        want = product(A[at], sa[at], B, sb, None if p is None else p[:, at])
        assert torch.equal(got[at], want)


@pytest.mark.parametrize("M,peers,tiles", [(16, 0, False), (16, 2, False), (300, 0, True), (300, 1, True)])
def test_columns_to_two_gibibytes(M, peers, tiles):
    N, K = 262_136, 8192                                 # B: 2^31 - 65536 bytes
    assert (gc.gemm_fp8_plan(M, N, K, peers)["tile_cols"] == 256) == tiles
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers}")
    A, sa, B, sb, p = exact_operands(M, N, K, peers, 2)
    got = gc.gemm_fp8(A, sa, B, sb, p)
    for j in (0, 1, 1023, 1024, 2046, 2047):
        at = slice(128 * j, min(128 * j + 128, N))
        want = product(A, sa, B[at], sb[j:j + 1], None if p is None else p[:, :, at])
        assert torch.equal(got[:, at], want)


@pytest.fixture(scope="module")
def room():
    """34 GB for nine blocks FAR apart."""
    return torch.empty(8 * FAR + (1 << 23), dtype=torch.bfloat16, device=DEV)


def apart(room, p):
    q = room.as_strided(p.shape, (FAR, p.shape[2], 1))
    q.copy_(p)
    return q


# streaming; tiles whose peers enter during the steps of K and after them; cut along K
@pytest.mark.parametrize("M,N,K,peers,which", [(20, 72, 400, 9, (16, 16)), (500, 4104, 656, 9, (64, "peers")),
                                               (1800, 2056, 1424, 3, (128, "peers")), (71, 5816, 8256, 3, (128, "cut"))])
def test_gemm_of_peers_far_apart(room, M, N, K, peers, which):
    assert instance(gc.gemm_fp8_plan(M, N, K, peers), peers) == which
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers} far apart")
    *ops, p = exact_operands(M, N, K, peers, 3)
    assert torch.equal(gc.gemm_fp8(*ops, apart(room, p)), product(*ops, p))


@pytest.mark.parametrize("M,N", [(3, 512), (5, 1024), (7, 4096), (9, 7168), (300, 7168), (2, 32768)])
def test_rms_norm_of_peers_far_apart(room, M, N):
    log(f"rms_norm M={M} N={N} peers far apart")
    x, p = torch.randn(M, N, device=DEV).bfloat16(), torch.randn(9, M, N, device=DEV).bfloat16()
    w = torch.randn(N, device=DEV)
    want = gc.rms_norm(x, w, partials=p, fp8=True)
    got = gc.rms_norm(x, w, partials=apart(room, p), fp8=True)
    assert torch.equal(got.y.view(torch.uint8), want.y.view(torch.uint8))
    assert torch.equal(got.scales, want.scales) and torch.equal(got.sum, want.sum)


def test_layer_of_peers_far_apart(room):
    T, E, K, F, N = 13, 12, 136, 72, 264
    x, lg = torch.randn(T, K, device=DEV).bfloat16(), torch.randn(T, E, device=DEV)
    w1, w2 = torch.randn(E, K, 2 * F, device=DEV).bfloat16(), torch.randn(E, F, N, device=DEV).bfloat16()
    p = torch.randn(9, T, N, device=DEV).bfloat16()
    assert torch.equal(gc.moe_layer(x, lg, w1, w2, 3, partials=apart(room, p)), gc.moe_layer(x, lg, w1, w2, 3, partials=p))
