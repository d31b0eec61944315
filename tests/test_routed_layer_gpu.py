"""examples/routed_layer.py: the projection, adapters, router, expert products
and combine in one pass, each stage within its bound of the 64-bit form of
the stage's own inputs, and the whole layer the same in every call."""
import importlib.util
import os

import pytest
import torch

import grouped_ref as ref
import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("routed_layer", os.path.join(ROOT, "examples", "routed_layer.py"))


@pytest.fixture(scope="module")
def ex():
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["routed_layer"] = m
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 37, 200])
def test_layer(ex, tokens):
    hidden, inner, experts, k, adapters, ranks = 264, 72, 10, 3, 4, 4
    log(f"layer of {tokens} tokens")
    p = ex.make_layer(hidden, inner, experts, adapters, 16, seed=tokens)
    x, ids, proj_peers, moe_peers = ex.make_batch(tokens, hidden, adapters, ranks, seed=tokens)
    groups = gc.group_rows(ids, adapters)
    out, r = ex.forward(p, x, groups, proj_peers, moe_peers, k, ranks)
    again, _ = ex.forward(p, x, groups, proj_peers, moe_peers, k, ranks)
    assert torch.equal(out, again)

    base = gc.gemm_ar(x, p.proj, proj_peers, R=ranks, rank=0)
    h = gc.lora_add(base, x, p.down, p.up, p.scale, groups.offsets, groups.rows)
    c = lambda t: t.cpu()  # noqa: E731
    ref.check(h, *ref.lora(c(base), c(x), c(p.down), c(p.up), c(p.scale), c(ids)), "adapters")
    want_ids, want_w = ref.route(c((h @ p.router).float()), k)
    assert torch.equal(c(r.ids), want_ids)
    assert torch.allclose(c(r.weights).double(), want_w, rtol=1e-5, atol=1e-30)
    a = gc.grouped_gemm(h, p.w1, r.offsets, r.rows, act="silu_glu")
    ref.check(a, *ref.grouped(c(h), c(p.w1), c(r.offsets), c(r.rows), "silu_glu"), "gate and up")
    y = gc.grouped_gemm(a, p.w2, r.offsets)
    ref.check(y, *ref.grouped(c(a), c(p.w2), c(r.offsets)), "down")
    ref.check(out, *ref.combine(c(y), c(r.slots), c(r.weights), c(moe_peers)), "combine")
