"""Routed and grouped operators beside the fused projections: binding of
include/gemm_coll_grouped.h.

    r = moe_route(logits, k)                          # ids, weights, offsets, rows, slots
    h = grouped_gemm(x, w_up, r.offsets, r.rows, act="silu_glu")
    y = grouped_gemm(h, w_down, r.offsets)
    out = moe_combine(y, r.slots, r.weights, partials)   # + the other ranks' partial sums

    g = group_rows(adapter_of_row, adapters)
    out = lora_add(out, x, down, up, scale, g.offsets, g.rows, out=out)

Tensors are on the current CUDA (HIP) device; calls are asynchronous on the
current stream (or ``stream=``).  Each (device, stream) pair gets its own
workspace, allocated on first use; pass ``workspace=`` (a zero-filled uint8
tensor) to use one of your own.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

import tensor_bf16_gemm_amd as _gc

__all__ = ["moe_route", "group_rows", "grouped_gemm", "moe_combine", "lora_add", "Routing", "Groups",
           "grouped_workspace_bytes", "lora_workspace_bytes"]

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


def declare(L: ctypes.CDLL) -> None:
    """Sets the signatures of the functions of include/gemm_coll_grouped.h."""
    i, i64, vp, u64 = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint64
    for name, args, res in (
            ("gemm_coll_grouped_workspace_bytes", [], i64),
            ("gemm_coll_lora_workspace_bytes", [i64, i], i64),
            ("gemm_coll_moe_route", [vp, i, i64, i64, i, i, i, vp, i, ctypes.c_float, vp, vp, vp, vp,
                                     vp, vp, u64, vp], i),
            ("gemm_coll_group_rows", [vp, i64, i, i, vp, vp, vp, vp, u64, vp], i),
            ("gemm_coll_grouped_gemm", [vp, i64, vp, vp, vp, i64, i64, i64, i, i, vp, vp, u64, vp], i),
            ("gemm_coll_moe_combine", [vp, i64, vp, vp, i64, i, i64, vp, i, i64, vp, vp], i),
            ("gemm_coll_lora_add", [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i, i, vp, vp, u64, vp], i)):
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res


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


def lora_workspace_bytes(M: int, r: int) -> int:
    """Bytes of workspace that lora_add needs for M rows and rank r on the current device."""
    n = _gc.lib().gemm_coll_lora_workspace_bytes(int(M), int(r))
    if n < 0:
        raise RuntimeError(f"gemm_coll_lora_workspace_bytes: {_gc.strerror(n)}")
    return n


def _workspace(workspace, stream: int, need: int) -> tuple[int | None, int]:
    """(pointer, bytes): None -> the (device, stream) pair's own of at least `need` bytes,
    False -> none, else the caller's."""
    if workspace is False:
        return None, 0
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    key = (torch.cuda.current_device(), stream)
    have = _scratch.get(key)
    if have is None or have[2] < need:
        # Twice what is asked for, so that growing sizes replace it seldom; a
        # replaced one stays allocated, for work in flight may still use it.
        n = need if have is None else max(need, 2 * have[2])
        t = torch.zeros(n, dtype=torch.uint8, device=f"cuda:{key[0]}")
        torch.cuda.synchronize(key[0])
        if have is not None:
            _kept.append(have[0])
        have = _scratch[key] = (t, t.data_ptr(), n)
    return have[1], have[2]


def _tensor(name, t, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _grouping(what, offsets, groups, rows=None, n=None):
    _tensor("offsets", offsets, torch.int32, (groups + 1,))
    if rows is not None:
        _tensor("rows", rows, torch.int32, None if n is None else (n,))
        if rows.dim() != 1:
            raise ValueError(f"{what}: rows must have one dimension")


def moe_route(logits, k: int, *, score: str = "softmax", bias=None, renormalize: bool = True,
              scale: float = 1.0, stream=None, workspace=None) -> Routing:
    """The k experts of largest logit (with ``bias`` [E]: of largest score + bias) for each row
    of logits [T,E] (float32 or bfloat16, rows may be strided), in falling order, lowest index
    first among equals; experts at -inf or NaN are never chosen (id -1, weight 0 where none is
    left).  weights: softmax over the row or sigmoid of the logit, divided by their sum with
    ``renormalize``, times ``scale``.  The T*k pairs come back grouped by expert."""
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16 [T, E], got {logits.dtype} {tuple(logits.shape)}")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    T, E = logits.shape
    if E > 1 and T > 0 and logits.stride(1) != 1:
        raise ValueError("logits: the experts of a row must be contiguous")
    if bias is not None:
        _tensor("bias", bias, torch.float32, (E,))
    dev = logits.device
    stride = logits.stride(0) if T > 1 else E
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    rows = torch.empty(T * k, dtype=torch.int32, device=dev)
    slots = torch.empty((T, k), dtype=torch.int32, device=dev)
    st = _gc._stream(stream)
    wp, wb = _workspace(workspace, st, grouped_workspace_bytes())
    _gc._check(_gc.lib().gemm_coll_moe_route(
        logits.data_ptr(), int(logits.dtype == torch.bfloat16), stride, T, E, k, _SCORES[score],
        None if bias is None else bias.data_ptr(), int(renormalize), scale, ids.data_ptr(),
        weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), wp, wb, st), "moe_route")
    return Routing(ids, weights, offsets, rows, slots)


def group_rows(ids, groups: int, *, stream=None, workspace=None) -> Groups:
    """Stable grouping of ids [T] or [T,k] (int32) into ``groups`` groups; ids outside
    [0, groups) are in none and come last.  rows[i] is the row (first index) of the item at
    position i, slots has the shape of ids."""
    if ids.dim() not in (1, 2):
        raise ValueError(f"ids must be [T] or [T, k], got {tuple(ids.shape)}")
    _tensor("ids", ids, torch.int32, None)
    T, k = ids.shape[0], ids.shape[1] if ids.dim() == 2 else 1
    offsets = torch.empty(groups + 1, dtype=torch.int32, device=ids.device)
    rows = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    slots = torch.empty_like(ids)
    st = _gc._stream(stream)
    wp, wb = _workspace(workspace, st, grouped_workspace_bytes())
    _gc._check(_gc.lib().gemm_coll_group_rows(ids.data_ptr(), T, k, groups, offsets.data_ptr(),
                                              rows.data_ptr(), slots.data_ptr(), wp, wb, st), "group_rows")
    return Groups(offsets, rows, slots)


def grouped_gemm(X, W, offsets, rows=None, out=None, *, act: str | None = None, stream=None,
                 workspace=None):
    """out[i] = X[rows[i]] . W[e] for offsets[e] <= i < offsets[e+1] (X[i] without rows), W
    [E,K,N]; act="silu_glu": silu of the first N/2 columns times the others, out [S,N/2].
    Positions in no group are left as they are.  workspace=False: no product is split along K."""
    if W.dim() != 3 or X.dim() != 2:
        raise ValueError(f"X must be [T, K] and W [E, K, N], got {tuple(X.shape)} and {tuple(W.shape)}")
    if act not in _ACTS:
        raise ValueError(f"act must be None or 'silu_glu', got {act!r}")
    T, K = X.shape
    E, _, N = W.shape
    _tensor("X", X, torch.bfloat16, None)
    _tensor("W", W, torch.bfloat16, (E, K, N))
    _grouping("grouped_gemm", offsets, E, rows)
    S = T if rows is None else rows.shape[0]
    F = N // 2 if act else N
    if out is None:
        out = torch.empty((S, F), dtype=torch.bfloat16, device=X.device)
    else:
        _tensor("out", out, torch.bfloat16, (S, F))
    st = _gc._stream(stream)
    wp, wb = _workspace(workspace, st, grouped_workspace_bytes())
    _gc._check(_gc.lib().gemm_coll_grouped_gemm(
        X.data_ptr(), T, W.data_ptr(), offsets.data_ptr(), None if rows is None else rows.data_ptr(),
        S, K, N, E, _ACTS[act], out.data_ptr(), wp, wb, st), "grouped_gemm")
    return out


def moe_combine(Y, slots, weights, partials=None, out=None, *, stream=None):
    """out [T,N] = bf16(sum over j of weights[t,j] * Y[slots[t,j]] + sum over p of partials[p,t]);
    slots outside Y (-1) are skipped.  partials [npeers,T,N] with contiguous rows; stride(0) may be
    larger (a row slice of every peer's partial, with the same slice of slots and weights)."""
    if Y.dim() != 2 or slots.dim() != 2:
        raise ValueError(f"Y must be [S, N] and slots [T, k], got {tuple(Y.shape)} and {tuple(slots.shape)}")
    S, N = Y.shape
    T, k = slots.shape
    _tensor("Y", Y, torch.bfloat16, None)
    _tensor("slots", slots, torch.int32, None)
    _tensor("weights", weights, torch.float32, (T, k))
    npeers, pp, stride = 0, None, 0
    if partials is not None and partials.shape[0] > 0:
        if partials.dtype != torch.bfloat16 or partials.dim() != 3 or partials.shape[1:] != (T, N):
            raise ValueError(f"partials: expected bf16 [npeers, {T}, {N}], got "
                             f"{partials.dtype} {tuple(partials.shape)}")
        if not partials.is_cuda:
            raise ValueError("partials must be a device tensor")
        if T * N > 0 and (partials.stride(2) != 1 or (T > 1 and partials.stride(1) != N)):
            raise ValueError("partials: rows must be contiguous")
        npeers, pp, stride = partials.shape[0], partials.data_ptr(), partials.stride(0)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=Y.device)
    else:
        _tensor("out", out, torch.bfloat16, (T, N))
    _gc._check(_gc.lib().gemm_coll_moe_combine(
        Y.data_ptr(), S, slots.data_ptr(), weights.data_ptr(), T, k, N, pp, npeers, stride,
        out.data_ptr(), _gc._stream(stream)), "moe_combine")
    return out


def lora_add(base, X, down, up, scale, offsets, rows, out=None, *, stream=None, workspace=None):
    """out [M,N] = bf16(base[m] + scale[a] * (X[m] . down[a]) . up[a]) for the rows m = rows[i] of
    adapter a's positions offsets[a] <= i < offsets[a+1] (group_rows of the rows' adapters), base[m]
    for rows of no adapter.  down [G,K,r], up [G,r,N], scale float32 [G]; out may be base."""
    if X.dim() != 2 or down.dim() != 3 or up.dim() != 3:
        raise ValueError("X must be [M, K], down [G, K, r] and up [G, r, N]")
    M, K = X.shape
    G, _, r = down.shape
    N = up.shape[2]
    _tensor("X", X, torch.bfloat16, None)
    _tensor("base", base, torch.bfloat16, (M, N))
    _tensor("down", down, torch.bfloat16, (G, K, r))
    _tensor("up", up, torch.bfloat16, (G, r, N))
    _tensor("scale", scale, torch.float32, (G,))
    _grouping("lora_add", offsets, G, rows, M)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    elif out is not base:
        _tensor("out", out, torch.bfloat16, (M, N))
    st = _gc._stream(stream)
    wp, wb = _workspace(workspace, st, grouped_workspace_bytes() + 4 * M * r + 512)
    _gc._check(_gc.lib().gemm_coll_lora_add(
        base.data_ptr(), X.data_ptr(), down.data_ptr(), up.data_ptr(), scale.data_ptr(),
        offsets.data_ptr(), rows.data_ptr(), M, K, N, r, G, out.data_ptr(), wp, wb, st), "lora_add")
    return out
