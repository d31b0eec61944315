"""The routers inside moe_layer: every kernel instance of them, more than 64
experts, and a bias for the selection, float32 and bfloat16."""
import math

import pytest
import torch

import layer_ref as ref
import tensor_bf16_gemm_amd as gc
from gpu_util import log
from test_layer_gpu import check_layer, dev, gen, layer_inputs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# What fp32 may move two keys of magnitude below 4 apart by: each is off by 2^-23 for the addition of
# the bias and, its score at most 1, 2^-24 times the 22 additions of a softmax's sum (16 in a lane, 6
# across the wave), the 16 of an exponent up to 16 and 6 of exp and the division.
KEYS = 2 * (2.0 ** -23 + (22 + 16 + 6) * 2.0 ** -24)


def apart(logits, k, score, bias):
    """Smallest distance between the keys of the last expert chosen and the first one left."""
    x = logits.double()
    key = (torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)) + bias.double()
    key = torch.where(x > -math.inf, key, -math.inf).sort(1, descending=True)[0]
    d = key[:, k - 1] - key[:, k]
    return float(d[torch.isfinite(d)].min())


# E 24, 64: 4 experts a lane; 80, 128, 256: 16 (vectors of them), 100, 250: single ones; 512, 1000: a wave a token
@pytest.mark.parametrize("E", [24, 64, 80, 100, 128, 250, 256, 512, 1000])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_layer_routes(E, dtype, score, biased):
    T, k = 13, 8
    log(f"moe_layer E={E} {dtype} {score} biased={biased}")
    ins = layer_inputs(T, E, k, 64, 32, 64, E, peers=1, dtype=dtype)
    ins[1][:, E // 3] = -math.inf                         # an expert out of service
    ins[1][4, 5:] = -math.inf                             # fewer experts than k
    bias = None
    if biased:
        bias = 0.3 * torch.randn(E, generator=gen(E + 1))
        assert apart(ins[1], k, score, bias) > KEYS
    check_layer(ins, k, score=score, bias=bias, renormalize=score == "sigmoid", scale=2.5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("first,local", [(0, 32), (100, 32), (224, 32)])
def test_layer_of_a_rank_of_256(dtype, first, local):
    """One rank's 32 of 256 experts under a biased sigmoid: the choice is over all of them."""
    ins = layer_inputs(16, 256, 8, 136, 72, 264, first, local=local, peers=2, dtype=dtype)
    bias = 0.3 * torch.randn(256, generator=gen(first + 1))
    assert apart(ins[1], 8, "sigmoid", bias) > KEYS
    ids, _ = ref.g.route(ins[1], 8, "sigmoid", bias)
    assert ((ids >= first) & (ids < first + local)).any()
    check_layer(ins, 8, first=first, score="sigmoid", bias=bias, scale=2.5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [128, 256, 250])
def test_layer_of_strided_logits(dtype, E):
    """Rows of logits inside a wider matrix, on and off the 16 bytes of a vector."""
    x, logits, w1, w2, _ = dev(*layer_inputs(9, E, 4, 64, 32, 64, E, dtype=dtype))
    want = gc.moe_layer(x, logits, w1, w2, 4)
    for ahead in (0, 1, 16):
        wide = torch.full((9, E + 32), math.nan, dtype=dtype, device="cuda")
        wide[:, ahead:ahead + E] = logits
        assert torch.equal(gc.moe_layer(x, wide[:, ahead:ahead + E], w1, w2, 4), want)
