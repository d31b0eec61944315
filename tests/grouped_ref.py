"""Plain 64-bit forms of the routed and grouped operators, on the CPU, and the
elementwise error bounds their tests use.

Bounds.  Products of bf16 values are exact in fp32.  A sum of n fp32 terms in
any order is off by at most (n + 2) u * sum|terms| (u = 2^-24, one u of slack
for each of two further roundings), and rounding y to bf16 (8 bits of
mantissa) by 2^-8 / (1 + 2^-8) |y|, or 2^-134 where y is that small.  What is composed (silu, the adapters' middle
activations) passes these on by its own derivative.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
BF = 2.0 ** -8
TINY = 2.0 ** -133


def group(ids, groups):
    """(offsets, rows, slots) of ids [T] or [T, k], one item after the other."""
    k = ids.shape[1] if ids.dim() == 2 else 1
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(groups + 1)]
    for i, g in enumerate(flat):
        lists[g if 0 <= g < groups else groups].append(i)
    offsets, rows, slots = [0], [], [-1] * len(flat)
    for g, items in enumerate(lists):
        for i in items:
            if g < groups:
                slots[i] = len(rows)
            rows.append(i // k)
        if g < groups:
            offsets.append(len(rows))
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(rows, dtype=i32),
            torch.tensor(slots, dtype=i32).reshape(ids.shape))


def route(logits, k, score="softmax", bias=None, renormalize=True, scale=1.0):
    """(ids, weights): k rounds of 'the largest that is left' in 64 bits."""
    x = logits.double()
    x = torch.where(torch.isnan(x), -torch.inf, x)
    T, E = x.shape
    if score == "softmax":
        high = x.amax(1, keepdim=True)
        e = torch.where(high == torch.inf, (x == torch.inf).double(), torch.exp(x - high))
        e = torch.where(x > -torch.inf, e, 0.0)
        s = e / e.sum(1, keepdim=True)
    else:
        s = torch.sigmoid(x)
    key = x.clone() if bias is None else torch.where(x > -torch.inf, s + bias.double(), -torch.inf)
    key = torch.where(torch.isnan(key), -torch.inf, key)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        left = key[t].tolist()
        for j in range(k):
            best = max(left)
            if best == -torch.inf:
                break
            at = left.index(best)
            ids[t, j], w[t, j] = at, s[t, at]
            left[at] = -torch.inf
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids, w * scale


def grouped(X, W, offsets, rows=None, act=None):
    """(values, bounds) of out [S, F]; rows of no group are NaN in both."""
    E, K, N = W.shape
    S = X.shape[0] if rows is None else rows.numel()
    F = N // 2 if act else N
    out = torch.full((S, F), torch.nan, dtype=torch.float64)
    tol = out.clone()
    off = offsets.tolist()
    for e in range(E):
        lo, hi = min(max(off[e], 0), S), min(max(off[e + 1], 0), S)
        if lo >= hi:
            continue
        at = torch.arange(lo, hi) if rows is None else rows[lo:hi].long()
        ok = (at >= 0) & (at < X.shape[0])
        x = torch.where(ok[:, None], X[at.clamp(0, max(X.shape[0] - 1, 0))].double(), 0.0)
        w = W[e].double()
        y, d = x @ w, (K + 2) * U * (x.abs() @ w.abs())
        if act:
            g, u, dg, du = y[:, :F], y[:, F:], d[:, :F], d[:, F:]
            s = g * torch.sigmoid(g)
            y = s * u
            # |silu'| <= 1.1; exp, the division and the products: 2^-19 of the value
            d = 1.1 * dg * (u.abs() + du) + s.abs() * du + 2.0 ** -19 * y.abs()
        out[lo:hi], tol[lo:hi] = y, d + BF * (y.abs() + d) + TINY
    return out, tol


def combine(Y, slots, weights, partials=None):
    T, k = slots.shape
    out = torch.zeros((T, Y.shape[1]), dtype=torch.float64)
    mag, n = out.clone(), k
    for j in range(k):
        ok = (slots[:, j] >= 0) & (slots[:, j] < Y.shape[0])
        term = torch.zeros_like(out)
        term[ok] = weights[ok, j, None].double() * Y[slots[ok, j].long()].double()
        out, mag = out + term, mag + term.abs()
    if partials is not None:
        n += partials.shape[0]
        out, mag = out + partials.double().sum(0), mag + partials.double().abs().sum(0)
    d = (n + 2) * U * mag
    return out, d + BF * (out.abs() + d) + TINY


def lora(base, X, down, up, scale, ids):
    out = base.double()
    tol = torch.zeros_like(out)
    K, r = down.shape[1:]
    for a in range(down.shape[0]):
        m = torch.nonzero(ids == a).flatten()
        if not len(m):
            continue
        x, D, V, s = X[m].double(), down[a].double(), up[a].double(), float(scale[a])
        h = s * (x @ D)
        # the fp32 sum and its scaling, then the two bf16 that carry it: 2^-16
        dh = (K + 3) * U * abs(s) * (x.abs() @ D.abs()) + 2.0 ** -16 * h.abs() + TINY
        out[m] += h @ V
        tol[m] = dh @ V.abs() + (2 * r + 4) * U * ((h.abs() + dh) @ V.abs() + base[m].double().abs())
    return out, torch.where(tol > 0, tol + BF * (out.abs() + tol) + TINY, 0.0)


def check(got, want, tol, what):
    """Every element within its bound; NaN bounds are not looked at."""
    look = ~torch.isnan(tol)
    g = got.double().cpu()
    bad = look & ~((g - want).abs() <= tol)
    if bad.any():
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(look.sum())} outside their bound; first "
                             f"{at}: got {float(g[at])!r}, want {float(want[at])!r} +- {float(tol[at])!r}")
