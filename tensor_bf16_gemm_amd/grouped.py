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
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32


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


# A call of a few microseconds feels every line of this module: the stream is
# read as its raw handle (a Stream object costs 2.7 us), and the checks are
# one expression per tensor that calls _refuse only to name what is wrong.

def _handle(stream) -> int:
    """hipStream_t of `stream`, None for the current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return _gc._stream(stream)


def _workspace(workspace, stream: int, more: int = 0) -> tuple[int | None, int]:
    """(pointer, bytes): None -> the (device, stream) pair's own, with at least `more` bytes
    beyond grouped_workspace_bytes(); False -> none; else the caller's."""
    if workspace is False:
        return None, 0
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    key = (torch._C._cuda_getDevice(), stream)
    have = _scratch.get(key)
    if have is None or have[2] < more:
        have = _new_scratch(key, have, more)
    return have[1], have[2] + _base_bytes[key[0]]


def _new_scratch(key, have, more):
    # Twice what is asked for, so that growing sizes replace it seldom; a
    # replaced one stays allocated, for work in flight may still use it.
    more = max(more, 2 * have[2]) if have else more
    t = torch.zeros(grouped_workspace_bytes() + more, dtype=torch.uint8, device=f"cuda:{key[0]}")
    torch.cuda.synchronize(key[0])
    if have:
        _kept.append(have[0])
    _scratch[key] = (t, t.data_ptr(), more)
    return _scratch[key]


def _refuse(name, t, dtype, shape=None):
    """Raises for what is wrong with the tensor."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def moe_route(logits, k: int, *, score: str = "softmax", bias=None, renormalize: bool = True,
              scale: float = 1.0, stream=None, workspace=None) -> Routing:
    """The k experts of largest logit (with ``bias`` [E]: of largest score + bias) for each row
    of logits [T,E] (float32 or bfloat16, rows may be strided), in falling order, lowest index
    first among equals; experts at -inf or NaN are never chosen (id -1, weight 0 where none is
    left).  weights: softmax over the row or sigmoid of the logit, divided by their sum with
    ``renormalize``, times ``scale``.  The T*k pairs come back grouped by expert."""
    dt = logits.dtype
    if logits.dim() != 2 or (dt is not _f32 and dt is not _bf16):
        raise TypeError(f"logits must be float32 or bfloat16 [T, E], got {dt} {tuple(logits.shape)}")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    T, E = logits.shape
    stride, step = logits.stride()
    if step != 1 and E > 1 and T > 0:
        raise ValueError("logits: the experts of a row must be contiguous")
    if T < 2:
        stride = E
    if bias is not None and not (bias.dtype is _f32 and bias.is_cuda and bias.is_contiguous()
                                 and bias.shape == (E,)):
        _refuse("bias", bias, _f32, (E,))
    dev = logits.device
    # one allocation for what has one entry per pair
    ids, slots, rows, weights = torch.empty(4, T, k, dtype=_i32, device=dev).unbind(0)
    rows, weights = rows.view(-1), weights.view(_f32)
    offsets = torch.empty(E + 1, dtype=_i32, device=dev)
    st = _handle(stream)
    wp, wb = _workspace(workspace, st)
    rc = _gc.lib().gemm_coll_moe_route(
        logits.data_ptr(), dt is _bf16, stride, T, E, k, _SCORES[score],
        None if bias is None else bias.data_ptr(), renormalize, scale, ids.data_ptr(),
        weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), wp, wb, st)
    if rc:
        _gc._check(rc, "moe_route")
    return Routing(ids, weights, offsets, rows, slots)


def group_rows(ids, groups: int, *, stream=None, workspace=None) -> Groups:
    """Stable grouping of ids [T] or [T,k] (int32) into ``groups`` groups; ids outside
    [0, groups) are in none and come last.  rows[i] is the row (first index) of the item at
    position i, slots has the shape of ids."""
    if ids.dim() not in (1, 2):
        raise ValueError(f"ids must be [T] or [T, k], got {tuple(ids.shape)}")
    if not (ids.dtype is _i32 and ids.is_cuda and ids.is_contiguous()):
        _refuse("ids", ids, _i32)
    T, k = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)
    offsets = torch.empty(groups + 1, dtype=_i32, device=ids.device)
    rows = torch.empty(T * k, dtype=_i32, device=ids.device)
    slots = torch.empty_like(ids)
    st = _handle(stream)
    wp, wb = _workspace(workspace, st)
    rc = _gc.lib().gemm_coll_group_rows(ids.data_ptr(), T, k, groups, offsets.data_ptr(),
                                        rows.data_ptr(), slots.data_ptr(), wp, wb, st)
    if rc:
        _gc._check(rc, "group_rows")
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
    E, KW, N = W.shape
    if not (X.dtype is _bf16 and X.is_cuda and X.is_contiguous()):
        _refuse("X", X, _bf16)
    if not (W.dtype is _bf16 and W.is_cuda and W.is_contiguous() and KW == K):
        _refuse("W", W, _bf16, (E, K, N))
    if not (offsets.dtype is _i32 and offsets.is_cuda and offsets.is_contiguous()
            and offsets.shape == (E + 1,)):
        _refuse("offsets", offsets, _i32, (E + 1,))
    S = T
    if rows is not None:
        if not (rows.dtype is _i32 and rows.is_cuda and rows.is_contiguous() and rows.dim() == 1):
            _refuse("rows", rows, _i32, "[S]")
        S = rows.shape[0]
    F = N // 2 if act else N
    if out is None:
        out = torch.empty(S, F, dtype=_bf16, device=X.device)
    elif not (out.dtype is _bf16 and out.is_cuda and out.is_contiguous() and out.shape == (S, F)):
        _refuse("out", out, _bf16, (S, F))
    st = _handle(stream)
    wp, wb = _workspace(workspace, st)
    rc = _gc.lib().gemm_coll_grouped_gemm(
        X.data_ptr(), T, W.data_ptr(), offsets.data_ptr(), None if rows is None else rows.data_ptr(),
        S, K, N, E, _ACTS[act], out.data_ptr(), wp, wb, st)
    if rc:
        _gc._check(rc, "grouped_gemm")
    return out


def moe_combine(Y, slots, weights, partials=None, out=None, *, stream=None):
    """out [T,N] = bf16(sum over j of weights[t,j] * Y[slots[t,j]] + sum over p of partials[p,t]);
    slots outside Y (-1) are skipped.  partials [npeers,T,N] with contiguous rows; stride(0) may be
    larger (a row slice of every peer's partial, with the same slice of slots and weights)."""
    if Y.dim() != 2 or slots.dim() != 2:
        raise ValueError(f"Y must be [S, N] and slots [T, k], got {tuple(Y.shape)} and {tuple(slots.shape)}")
    S, N = Y.shape
    T, k = slots.shape
    if not (Y.dtype is _bf16 and Y.is_cuda and Y.is_contiguous()):
        _refuse("Y", Y, _bf16)
    if not (slots.dtype is _i32 and slots.is_cuda and slots.is_contiguous()):
        _refuse("slots", slots, _i32)
    if not (weights.dtype is _f32 and weights.is_cuda and weights.is_contiguous()
            and weights.shape == (T, k)):
        _refuse("weights", weights, _f32, (T, k))
    npeers, pp, stride = 0, None, 0
    if partials is not None and partials.shape[0] > 0:
        if not (partials.dtype is _bf16 and partials.dim() == 3 and partials.shape[1:] == (T, N)):
            raise ValueError(f"partials: expected bf16 [npeers, {T}, {N}], got "
                             f"{partials.dtype} {tuple(partials.shape)}")
        if not partials.is_cuda:
            raise ValueError("partials must be a device tensor")
        stride, by_row, by_col = partials.stride()
        if T * N > 0 and (by_col != 1 or (T > 1 and by_row != N)):
            raise ValueError("partials: rows must be contiguous")
        npeers, pp = partials.shape[0], partials.data_ptr()
    if out is None:
        out = torch.empty(T, N, dtype=_bf16, device=Y.device)
    elif not (out.dtype is _bf16 and out.is_cuda and out.is_contiguous() and out.shape == (T, N)):
        _refuse("out", out, _bf16, (T, N))
    rc = _gc.lib().gemm_coll_moe_combine(
        Y.data_ptr(), S, slots.data_ptr(), weights.data_ptr(), T, k, N, pp, npeers, stride,
        out.data_ptr(), _handle(stream))
    if rc:
        _gc._check(rc, "moe_combine")
    return out


def lora_add(base, X, down, up, scale, offsets, rows, out=None, *, stream=None, workspace=None):
    """out [M,N] = bf16(base[m] + scale[a] * (X[m] . down[a]) . up[a]) for the rows m = rows[i] of
    adapter a's positions offsets[a] <= i < offsets[a+1] (group_rows of the rows' adapters), base[m]
    for rows of no adapter.  down [G,K,r], up [G,r,N], scale float32 [G]; out may be base."""
    if X.dim() != 2 or down.dim() != 3 or up.dim() != 3:
        raise ValueError("X must be [M, K], down [G, K, r] and up [G, r, N]")
    M, K = X.shape
    G, KD, r = down.shape
    N = up.shape[2]
    if not (X.dtype is _bf16 and X.is_cuda and X.is_contiguous()):
        _refuse("X", X, _bf16)
    if not (base.dtype is _bf16 and base.is_cuda and base.is_contiguous() and base.shape == (M, N)):
        _refuse("base", base, _bf16, (M, N))
    if not (down.dtype is _bf16 and down.is_cuda and down.is_contiguous() and KD == K):
        _refuse("down", down, _bf16, (G, K, r))
    if not (up.dtype is _bf16 and up.is_cuda and up.is_contiguous() and up.shape == (G, r, N)):
        _refuse("up", up, _bf16, (G, r, N))
    if not (scale.dtype is _f32 and scale.is_cuda and scale.is_contiguous() and scale.shape == (G,)):
        _refuse("scale", scale, _f32, (G,))
    if not (offsets.dtype is _i32 and offsets.is_cuda and offsets.is_contiguous()
            and offsets.shape == (G + 1,)):
        _refuse("offsets", offsets, _i32, (G + 1,))
    if not (rows.dtype is _i32 and rows.is_cuda and rows.is_contiguous() and rows.shape == (M,)):
        _refuse("rows", rows, _i32, (M,))
    if out is None:
        out = torch.empty(M, N, dtype=_bf16, device=X.device)
    elif out is not base and not (out.dtype is _bf16 and out.is_cuda and out.is_contiguous()
                                  and out.shape == (M, N)):
        _refuse("out", out, _bf16, (M, N))
    st = _handle(stream)
    wp, wb = _workspace(workspace, st, 4 * M * r if M * r > 1 << 20 else 0)
    rc = _gc.lib().gemm_coll_lora_add(
        base.data_ptr(), X.data_ptr(), down.data_ptr(), up.data_ptr(), scale.data_ptr(),
        offsets.data_ptr(), rows.data_ptr(), M, K, N, r, G, out.data_ptr(), wp, wb, st)
    if rc:
        _gc._check(rc, "lora_add")
    return out
