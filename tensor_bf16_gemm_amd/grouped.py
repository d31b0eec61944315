"""Routed and grouped operators beside the fused projections: binding of
include/gemm_coll_grouped.h.

    r = moe_route(logits, k)                          # ids, weights, offsets, rows, slots
    h = grouped_gemm(x, w_up, r.offsets, r.rows, act="silu_glu")
    y = grouped_gemm(h, w_down, r.offsets)
    out = moe_combine(y, r.slots, r.weights, partials)   # + the other ranks' partial sums

    # with the experts first .. first + local - 1 on this rank: the others' pairs get slot -1
    g = group_rows(r.ids - first, local)
    h = grouped_gemm(x, w_up[local ones], g.offsets, g.rows, act="silu_glu")
    out = moe_combine(grouped_gemm(h, w_down[local ones], g.offsets), g.slots, r.weights, partials)

    g = group_rows(adapter_of_row, adapters)
    out = lora_add(out, x, down, up, scale, g.offsets, g.rows, out=out)

Tensors are on the current CUDA (HIP) device; calls are asynchronous on the
current stream (or ``stream=``, as for the package's other calls).  Each (device, stream) pair gets its own
workspace, allocated on first use; pass ``workspace=`` (a zero-filled uint8
tensor) to use one of your own.  A captured graph keeps the workspace of the
stream it was captured on: replay it on that stream, or while nothing else
runs there.

The tensors are checked, the outputs made and the library called in the
extension module _native (csrc/binding.cpp); these functions add the stream,
the workspace and the names.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

import tensor_bf16_gemm_amd as _gc
from tensor_bf16_gemm_amd.grouped_abi import GroupedPlan

try:
    from . import _native
except ImportError as e:
    raise RuntimeError("tensor_bf16_gemm_amd/_native.so is missing or does not load: build it with "
                       "`python -m tensor_bf16_gemm_amd.build`") from e

__all__ = ["moe_route", "group_rows", "grouped_gemm", "moe_combine", "lora_add", "Routing", "Groups",
           "grouped_plan", "grouped_workspace_bytes", "lora_workspace_bytes"]

_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTS = {None: 0, "silu_glu": 1}


class Routing(NamedTuple):
    """ids, weights [T,k]; offsets [E+1], rows [T*k], slots [T,k]: the pairs grouped by expert."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


class Groups(NamedTuple):
    """offsets [groups+1], rows (row of each position), slots (position of each item)."""
    offsets: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


_base_bytes: dict[int, int] = {}
_scratch: dict[tuple[int, int], tuple[torch.Tensor, int, int]] = {}
_kept: list[torch.Tensor] = []


def grouped_workspace_bytes() -> int:
    """Bytes of workspace that lets any call here but lora_add run on the current device."""
    dev = torch.cuda.current_device()
    n = _base_bytes.get(dev)
    if n is None:
        n = _gc.lib().gemm_coll_grouped_workspace_bytes()
        if n < 0:
            raise RuntimeError(f"gemm_coll_grouped_workspace_bytes: {_gc.strerror(n)}")
        _base_bytes[dev] = n
    return n


def grouped_plan(S: int, K: int, N: int, E: int, *, act: str | None = None, workspace: bool = True,
                 cus: int = 256) -> dict:
    """How grouped_gemm runs S rows in E groups (host arithmetic only, no GPU needed)."""
    pl = GroupedPlan()
    rc = _gc.lib().gemm_coll_grouped_plan(S, K, N, E, _ACTS[act], int(workspace), cus, ctypes.byref(pl))
    _gc._check(rc, "grouped_plan")
    return {n: int(getattr(pl, n)) for n, _ in GroupedPlan._fields_}


def lora_workspace_bytes(M: int, r: int) -> int:
    """Bytes of workspace that lora_add needs for M rows and rank r on the current device."""
    n = _gc.lib().gemm_coll_lora_workspace_bytes(int(M), int(r))
    if n < 0:
        raise RuntimeError(f"gemm_coll_lora_workspace_bytes: {_gc.strerror(n)}")
    return n


def _handle(stream) -> int:
    """hipStream_t of `stream`, None for the current one (read as the raw handle: a Stream
    object costs 2.7 us, as much as a kernel launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return _gc._stream(stream)


def _workspace(workspace, stream: int, more: int = 0) -> tuple[int | None, int]:
    """(pointer, bytes): None -> the (device, stream) pair's own, with at least `more` bytes
    beyond grouped_workspace_bytes(); False -> none; else the caller's."""
    if workspace is False:
        return None, 0
    if workspace is not None:
        return _gc._own_workspace(workspace)
    key = (torch._C._cuda_getDevice(), stream)
    have = _scratch.get(key)
    if have is None or have[2] < more:
        have = _new_scratch(key, more)
    return have[1], have[2] + _base_bytes[key[0]]


def _new_scratch(key, more):
    # One thread at a time (the synchronization lets others run), and the next
    # finds what this one has made.  At least twice the size of the one before,
    # so that growing sizes replace it seldom; a replaced one stays allocated,
    # for work in flight may still use it.
    with _gc._making:
        have = _scratch.get(key)
        if have is not None and have[2] >= more:
            return have
        more = max(more, 2 * have[2]) if have else more
        t = torch.zeros(grouped_workspace_bytes() + more, dtype=torch.uint8, device=f"cuda:{key[0]}")
        torch.cuda.synchronize(key[0])
        if have:
            _kept.append(have[0])
        _scratch[key] = (t, t.data_ptr(), more)
        return _scratch[key]


def _place(t, workspace, more: int = 0, stream=None):
    """(stream, workspace, bytes) for a call on tensor t; nothing is set up for a host tensor,
    which the call refuses."""
    if not t.is_cuda:
        return 0, None, 0
    st = _handle(stream)
    return st, *_workspace(workspace, st, more)


def _on(stream, call, *args):
    """call(*args) for a launch on `stream`.  On a stream that is not the current one the outputs
    come from its memory, and the inputs' is kept until it is through with them."""
    side = None if stream is None else _gc._side(stream)
    if side is None:
        return call(*args)
    with torch.cuda.stream(side):
        r = call(*args)
    here = torch.cuda.current_stream()
    for t in r if isinstance(r, tuple) else (r,):
        t.record_stream(here)
    _gc._hold(stream, *(t for t in args if isinstance(t, torch.Tensor)))
    return r


def moe_route(logits, k: int, *, score: str = "softmax", bias=None, renormalize: bool = True,
              scale: float = 1.0, stream=None, workspace=None) -> Routing:
    """The k experts of largest logit (with ``bias`` [E]: of largest score + bias) for each row
    of logits [T,E] (float32 or bfloat16, rows may be strided), in falling order, lowest index
    first among equals; experts at -inf or NaN are never chosen (id -1, weight 0 where none is
    left).  weights: softmax over the row or sigmoid of the logit, divided by their sum with
    ``renormalize``, times ``scale``.  The T*k pairs come back grouped by expert."""
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return Routing._make(_on(stream, _native.moe_route, logits, k, _SCORES[score], bias, renormalize, scale,
                             *_place(logits, workspace, 0, stream)))


def group_rows(ids, groups: int, *, stream=None, workspace=None) -> Groups:
    """Stable grouping of ids [T] or [T,k] (int32) into ``groups`` groups; ids outside
    [0, groups) are in none and come last.  rows[i] is the row (first index) of the item at
    position i, slots has the shape of ids."""
    return Groups._make(_on(stream, _native.group_rows, ids, groups, *_place(ids, workspace, 0, stream)))


def grouped_gemm(X, W, offsets, rows=None, out=None, *, act: str | None = None, stream=None,
                 workspace=None):
    """out[i] = X[rows[i]] . W[e] for offsets[e] <= i < offsets[e+1] (X[i] without rows), W
    [E,K,N]; act="silu_glu": silu of the first N/2 columns times the others, out [S,N/2].
    Positions in no group are left as they are.  workspace=False: no product is split along K."""
    if act not in _ACTS:
        raise ValueError(f"act must be None or 'silu_glu', got {act!r}")
    return _on(stream, _native.grouped_gemm, X, W, offsets, rows, out, _ACTS[act],
               *_place(X, workspace, 0, stream))


def moe_combine(Y, slots, weights, partials=None, out=None, *, stream=None):
    """out [T,N] = bf16(sum over j of weights[t,j] * Y[slots[t,j]] + sum over p of partials[p,t]);
    slots outside Y (-1) are skipped.  partials [npeers,T,N] with contiguous rows; stride(0) may be
    larger (a row slice of every peer's partial, with the same slice of slots and weights)."""
    return _on(stream, _native.moe_combine, Y, slots, weights, partials, out,
               _handle(stream) if Y.is_cuda else 0)


def lora_add(base, X, down, up, scale, offsets, rows, out=None, *, stream=None, workspace=None):
    """out [M,N] = bf16(base[m] + scale[a] * (X[m] . down[a]) . up[a]) for the rows m = rows[i] of
    adapter a's positions offsets[a] <= i < offsets[a+1] (group_rows of the rows' adapters), base[m]
    for rows of no adapter.  down [G,K,r], up [G,r,N], scale float32 [G]; out may be base."""
    sums = X.shape[0] * down.shape[-1]               # fp32, in the workspace
    return _on(stream, _native.lora_add, base, X, down, up, scale, offsets, rows, out,
               *_place(X, workspace, 4 * sums if sums > 1 << 24 else 0, stream))
