"""Operators between and around the projections of a layer: binding of
include/gemm_coll_layer.h.

    n = rms_norm(x, weight, residual=h, partials=peers, fp8=True)   # n.y e4m3, n.scales, n.sum
    out = gemm_fp8(n.y, n.scales, wq, wq_scales, partials)          # projection + the other ranks' partials
    wq, wq_scales = quantize_fp8(w, block_rows=128)                 # w [N,K], once
    out = moe_layer(x, logits, w1, w2, k, partials=partials)        # up to 16 tokens

Tensors, streams, workspaces and errors are as in .grouped, whose workspace
these calls share.  Forward only: outputs carry no gradient, also of inputs that
require one.  A row's result may differ in its last places (a code by one) with
the number of rows of the call, whose kernel decides the order of its sums.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

import tensor_bf16_gemm_amd as _gc
from tensor_bf16_gemm_amd.grouped import _SCORES, _handle, _native, _on, _place
from tensor_bf16_gemm_amd.layer_abi import Fp8Plan

__all__ = ["rms_norm", "quantize_fp8", "gemm_fp8", "moe_layer", "Norm", "Quantized", "gemm_fp8_plan"]


class Norm(NamedTuple):
    """y [M,N] bf16 or e4m3; scales [M,ceil(N/128)] of e4m3, else None; sum [M,N]: x with the
    residual and the partials, None where there are neither."""
    y: torch.Tensor
    scales: torch.Tensor | None
    sum: torch.Tensor | None


class Quantized(NamedTuple):
    """q [M,K] e4m3, scales float32 [M,ceil(K/128)] or [ceil(M/128),ceil(K/128)]."""
    q: torch.Tensor
    scales: torch.Tensor


def rms_norm(x, weight, *, residual=None, partials=None, eps: float = 1e-6, fp8: bool = False, out=None,
             scales=None, sum_out=None, stream=None) -> Norm:
    """h = x + residual + sum over p of partials[p] (fp32), y = h / sqrt(mean(h^2) + eps) * weight for
    the rows of x [M,N] bf16.  weight [N] bf16 or float32; partials [npeers,M,N], as for moe_combine.
    y is bf16, or with ``fp8`` e4m3 with a scale per row and 128 columns.  sum is bf16(h); sum_out may
    be x or residual, and out (bf16) x or residual where sum_out is another."""
    return Norm._make(_on(stream, _native.rms_norm, x, weight, residual, partials, eps, fp8, out, scales, sum_out,
                          _handle(stream) if x.is_cuda else 0))


def quantize_fp8(x, *, block_rows: int = 1, out=None, scales=None, stream=None) -> Quantized:
    """e4m3 codes of x [M,K] bf16 with a scale per row and 128 columns (block_rows=1) or per 128 x 128
    block (block_rows=128): scale = max(largest |value|, 2^-100) / 448.  A block with an infinity or
    a NaN gets NaN for its scale and codes."""
    return Quantized._make(_on(stream, _native.quantize_fp8, x, block_rows, out, scales,
                               _handle(stream) if x.is_cuda else 0))


def gemm_fp8(A, a_scales, B, b_scales, partials=None, out=None, *, stream=None, workspace=None):
    """out [M,N] = bf16(sum over the blocks b of 128 of K of a_scales[m,b] * b_scales[n//128,b] *
    A[m,b] . B[n,b] + sum over p of partials[p]) for e4m3 A [M,K] and B [N,K].  a_scales float32
    [M,ceil(K/128)] with any strides (contiguous columns, as quantize_fp8 and rms_norm return them, are
    best for few rows; where gemm_fp8_plan gives tiles of 256 columns, contiguous rows, as of
    a_scales.t().contiguous().t(), save up to 7 %); b_scales float32 [ceil(N/128),ceil(K/128)];
    partials [npeers,M,N], as for moe_combine.  workspace=False: no product is split along K."""
    return _on(stream, _native.gemm_fp8, A, a_scales, B, b_scales, partials, out, *_place(A, workspace, 0, stream))


def gemm_fp8_plan(M: int, N: int, K: int, npeers: int = 0, *, workspace: bool = True, cus: int = 256) -> dict:
    """How gemm_fp8 runs these sizes (host arithmetic only, no GPU needed)."""
    pl = Fp8Plan()
    _gc._check(_gc.lib().gemm_coll_gemm_fp8_plan(M, N, K, npeers, int(workspace), cus, ctypes.byref(pl)),
               "gemm_fp8_plan")
    return {n: int(getattr(pl, n)) for n, _ in Fp8Plan._fields_}


def moe_layer(x, logits, w1, w2, k: int, *, first: int = 0, score: str = "softmax", bias=None,
              renormalize: bool = True, scale: float = 1.0, partials=None, out=None, stream=None,
              workspace=None):
    """A layer of experts for x [T,K], T at most 16, in two launches: the k experts of each token as
    moe_route chooses them from logits [T,E] (score, bias, renormalize, scale likewise), and
    out [T,N] = bf16(sum over the chosen experts that are here of weight * (a . w2[e - first]) + sum
    over p of partials[p]), a = bf16(silu(g) * u), (g, u) the halves of x . w1[e - first].  w1
    [local,K,2F] and w2 [local,F,N] hold the experts first .. first + local - 1 of the E; an expert
    that a token has not chosen does not touch its row, whatever its weights hold."""
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _on(stream, _native.moe_layer, x, logits, w1, w2, k, _SCORES[score], bias, renormalize, scale, first,
               partials, out, *_place(x, workspace, 0, stream))
