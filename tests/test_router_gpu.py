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


def check_routing(logits, k, workspace=None, **kw):
    T, E = logits.shape
    log(f"route T={T} E={E} k={k} {logits.dtype} workspace={workspace}")
    r = gc.moe_route(logits.to(DEV), k, workspace=workspace, **kw)
    ids, w = ref.route(logits, k, **kw)
    assert torch.equal(r.ids.cpu(), ids)
    # exp and the division: a few units; x - max rounds by |x - max| u; the sum by E u
    bound = (2 * float(logits.float().abs().max()) + E + 32) * 2 * ref.U
    assert torch.all((r.weights.cpu().double() - w).abs() <= bound * w.abs() + 1e-37)
    for got, want, name in zip((r.offsets, r.rows, r.slots), ref.group(ids, E), ("offsets", "rows", "slots")):
        assert torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("T,E,k", [(129, 64, 1), (1024, 20, 1), (33, 257, 8), (341, 300, 3), (146, 5, 7)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_without_workspace(T, E, k, dtype):
    """More tokens than one workgroup routes at a time, in one workgroup."""
    logits = (torch.randn((T, E), generator=gen(T)) * 2).to(dtype)
    check_routing(logits, k, workspace=False)
    check_routing(logits, k, score="sigmoid")


def test_renormalize_without_a_truth_value_is_refused():
    class Neither:
        def __bool__(self):
            raise ValueError("neither true nor false")
    with pytest.raises(ValueError, match="neither"):
        gc.moe_route(torch.zeros((2, 4), device=DEV), 2, renormalize=Neither())
    with pytest.raises(TypeError):
        gc.moe_route(torch.zeros((2, 4), device=DEV), 2, scale="1")


@pytest.mark.parametrize("T,E,k", [(16500, 24, 2), (17000, 60, 1), (4200, 300, 3), (4100, 600, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_blocks_of_several_passes(T, E, k, dtype):
    """Blocks of more tokens than a workgroup routes at a time (64, or 16 with more than 256 experts)."""
    logits = (torch.randn((T, E), generator=gen(T)) * 2).to(dtype)
    check_routing(logits, k, score="sigmoid", scale=2.5)


@pytest.mark.parametrize("E,k", [(48, 4), (300, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bias_chooses_experts_far_below_the_maximum(E, k, dtype):
    """Softmax, renormalized over the chosen: their weights depend on the chosen logits alone, however
    small their scores are."""
    g = gen(E)
    x = torch.randn((9, E), generator=g)
    x[:, 5] += torch.linspace(0, 400, 9)              # the maximum, which the bias keeps out
    bias = 2.0 * torch.randperm(E, generator=g).float()
    bias[5] = -10.0
    x = x.to(dtype)
    ids, w = ref.route(x, k, bias=bias)
    r = gc.moe_route(x.to(DEV), k, bias=bias.to(DEV))
    log(f"route with bias E={E} {dtype}")
    assert torch.equal(r.ids.cpu(), ids)
    # differences of the chosen logits (below 10 here) round by u each, exp and the division by a few
    assert torch.all((r.weights.cpu().double() - w).abs() <= (10 + 32) * 2 * ref.U * w)
