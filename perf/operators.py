"""Cases, plain forms and exact values of the routed and grouped operators.

Four operators of a tensor- or expert-parallel transformer layer, beside the
projections of this package:

  route    moe_route: top-k choice of experts for every token, its weights,
           and the grouping of the chosen (token, expert) pairs by expert
  experts  grouped_gemm: one matrix product per expert, ragged row counts,
           optionally gathering its rows and ending in silu(gate) * up
  combine  moe_combine: the weighted sum of every token's expert rows, plus
           the other ranks' partial sums
  lora     lora_add: low-rank adapters of many requests beside a projection

Hidden sizes 7168 and 6288 / 3648, the 896 = 7168 / 8 columns of one of
eight ranks, and up to 7 peers are the sizes of workloads/; expert counts,
ranks of adapters and token counts are generic.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One decode step of a batch of 64 requests: the smallest router call,
        # where latency is all there is.
        dict(name="route_decode", op="route", T=64, E=64, k=8, dtype="f32", score="softmax",
             renorm=True, masked=0.0),
        # A prefill chunk over many experts, bf16 logits (ties are common) and
        # experts taken out of service.
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, dtype="bf16", score="sigmoid",
             renorm=True, masked=0.1),
        # One request, one token: gate and up products of 8 of 64 experts.
        dict(name="up_token", op="experts", T=1, k=8, E=64, K=7168, N=1792, glu=True, gather=True,
             skew=0.0),
        # A decode batch: every expert is read, about 8 rows each.
        dict(name="up_decode", op="experts", T=64, k=8, E=64, K=7168, N=1792, glu=True,
             gather=True, skew=1.0),
        # A mixed batch, odd sizes, skewed experts, about 116 rows each.
        dict(name="down_odd", op="experts", T=777, k=6, E=40, K=904, N=3648, glu=False,
             gather=False, skew=1.5),
        # A prefill chunk: gate and up products, 512 rows an expert on average.
        dict(name="up_prefill", op="experts", T=4096, k=8, E=64, K=7168, N=1792, glu=True,
             gather=True, skew=0.5),
        # The down products of a prefill chunk twice as long: short K, wide
        # output, the largest case.
        dict(name="down_prefill", op="experts", T=8192, k=8, E=64, K=896, N=7168, glu=False,
             gather=False, skew=0.5),
        # A small decode batch where half of the experts live on other ranks.
        dict(name="combine_decode", op="combine", T=16, k=8, N=7168, peers=7, local=0.5),
        # A prefill chunk: every chosen expert is here, 7 peers hold partials.
        dict(name="combine_prefill", op="combine", T=4096, k=8, N=7168, peers=7, local=1.0),
        # One token with one adapter.
        dict(name="lora_token", op="lora", M=1, K=7168, N=6288, r=16, G=8, none=0.0),
        # A decode batch whose requests use 32 adapters, some of them none.
        dict(name="lora_decode", op="lora", M=64, K=7168, N=6288, r=32, G=32, none=0.1),
        # A prefill batch of a few long requests.
        dict(name="lora_prefill", op="lora", M=4096, K=7168, N=6288, r=64, G=8, none=0.1),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, -(-lo // step) * step), hi // step * step)
    return v + step if v == 3 * 1024 else v


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "experts", "combine", "lora", "lora"])
    if op == "route":
        E = _spread(rng, 8, 512)
        return dict(op=op, T=_spread(rng, 1, 16384), E=E, k=rng.randint(1, 8),
                    dtype=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.7, masked=rng.choice([0.0, 0.0, 0.2]))
    if op == "experts":
        glu, E = rng.random() < 0.5, _spread(rng, 4, 64)
        k = rng.randint(1, min(8, E))
        K, N = _spread(rng, 256, 7168, 8), _spread(rng, 256, 7168, 16 if glu else 8)
        # no more weights than up_decode has, no more products than up_prefill
        while E * K * N > 64 * 7168 * 1792:
            K, N = max(256, K // 16 * 8), max(256, N // 32 * 16)
        T = _spread(rng, 1, max(1, min(4096, int(4096 * 8 * 7168 * 1792 / (k * K * N)))))
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, glu=glu, gather=rng.random() < 0.5,
                    skew=rng.choice([0.0, 0.5, 1.5]))
    if op == "combine":
        return dict(op=op, T=_spread(rng, 1, 4096), k=rng.randint(1, 8),
                    N=_spread(rng, 256, 7168, 8), peers=rng.randint(0, 7),
                    local=rng.choice([1.0, 0.5, 0.125]))
    return dict(op=op, M=_spread(rng, 1, 4096), K=_spread(rng, 256, 7168, 8),
                N=_spread(rng, 256, 6288, 8), r=_spread(rng, 8, 64, 8), G=_spread(rng, 1, 64),
                none=rng.choice([0.0, 0.1, 0.5]))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    x = torch.randn(shape, generator=g, dtype=dtype, device=DEV)
    return x.mul_(scale) if scale != 1.0 else x


def _group(ids, groups):
    """offsets, rows and slots of the stable grouping of ids (flat, of k a token)."""
    k = ids.shape[1] if ids.dim() == 2 else 1
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= groups), groups, flat)
    by, order = torch.sort(key, stable=True)
    bounds = torch.arange(groups + 1, device=ids.device)
    offsets = torch.searchsorted(by, bounds).int()
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=ids.device)
    slots = torch.where(key == groups, -1, slots).int().reshape(ids.shape)
    return offsets, (order // k).int(), slots


def _choose(g, T, k, E, skew):
    """k distinct experts for each of T tokens, some experts more often."""
    x = torch.randn((T, E), generator=g, device=DEV)
    x += skew * torch.randn((1, E), generator=g, device=DEV)
    return torch.sort(x, dim=1, descending=True).indices[:, :k].int()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if s["op"] == "route":
        x = _randn(g, s["T"], s["E"], dtype=torch.float32)
        if s["masked"] > 0:
            out = torch.rand((1, s["E"]), generator=g, device=DEV) < s["masked"]
            x = x.masked_fill(out, -math.inf)
            if s["T"] > 1:
                x[s["T"] // 2] = -math.inf      # a padding token: no expert at all
        s["logits"] = x.bfloat16() if s["dtype"] == "bf16" else x
    elif s["op"] == "experts":
        ids = _choose(g, s["T"], s["k"], s["E"], s["skew"])
        s["offsets"], rows, _ = _group(ids, s["E"])
        s["rows"] = rows if s["gather"] else None
        s["X"] = _randn(g, s["T"] if s["gather"] else s["T"] * s["k"], s["K"])
        s["W"] = _randn(g, s["E"], s["K"], s["N"], scale=s["K"] ** -0.5)
        sizes = (s["offsets"][1:] - s["offsets"][:-1]).long()
        s["active"] = torch.nonzero(sizes).flatten()
        s["most"] = int(sizes.max())
    elif s["op"] == "combine":
        flat = torch.rand(s["T"] * s["k"], generator=g, device=DEV) < s["local"]
        flat[0] = True
        order = torch.argsort(torch.rand(flat.numel(), generator=g, device=DEV))
        here = order[flat[order]]                 # the pairs with an expert here, shuffled
        slots = torch.full((s["T"] * s["k"],), -1, dtype=torch.int32, device=DEV)
        slots[here] = torch.arange(here.numel(), dtype=torch.int32, device=DEV)
        s["slots"] = slots.reshape(s["T"], s["k"])
        s["Y"] = _randn(g, here.numel(), s["N"])
        w = torch.rand((s["T"], s["k"]), generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["partials"] = _randn(g, s["peers"], s["T"], s["N"]) if s["peers"] else None
    else:
        ids = torch.randint(0, s["G"], (s["M"],), generator=g, device=DEV, dtype=torch.int32)
        ids[torch.rand(s["M"], generator=g, device=DEV) < s["none"]] = -1
        s["offsets"], s["rows"], _ = _group(ids, s["G"])
        s["ids"] = ids
        s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
        s["n"] = int(s["offsets"][-1])           # rows with an adapter
        s["X"] = _randn(g, s["M"], s["K"])
        s["base"] = _randn(g, s["M"], s["N"])
        s["down"] = _randn(g, s["G"], s["K"], s["r"], scale=s["K"] ** -0.5)
        s["up"] = _randn(g, s["G"], s["r"], s["N"], scale=s["r"] ** -0.5)
        s["scale"] = torch.rand(s["G"], generator=g, device=DEV) + 0.5
    return s


def _padded(offsets, most, n):
    """Positions [groups, most] of every group's rows; those past its end hold others of the n."""
    return (offsets[:-1, None].long() + torch.arange(most, device=offsets.device)).clamp(max=n - 1)


def _places(offsets, n):
    """The group of every position below n, and the position's place in its group."""
    at = torch.arange(n, device=offsets.device)
    group = torch.searchsorted(offsets[1:], at.int(), right=True)
    return group, at - offsets[group]


def _route(s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    k = min(s["k"], s["E"])
    top, ids = top[:, :k], ids[:, :k]
    chosen = top > -math.inf
    if s["score"] == "softmax":
        high = x.amax(1, keepdim=True)
        w = torch.exp(top - high) / torch.exp(x - high).sum(1, keepdim=True)
    else:
        w = 1.0 / (1.0 + torch.exp(-top))
    w = torch.where(chosen, w, 0.0)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    ids = torch.where(chosen, ids, -1).int()
    if k < s["k"]:                               # more places than experts
        ids = torch.nn.functional.pad(ids, (0, s["k"] - k), value=-1)
        w = torch.nn.functional.pad(w, (0, s["k"] - k))
    offsets, rows, slots = _group(ids, s["E"])
    return dict(ids=ids, weights=w, offsets=offsets, rows=rows, slots=slots)


def _experts(s):
    n = s["T"] * s["k"]
    at = _padded(s["offsets"], s["most"], n)[s["active"]]
    if s["rows"] is not None:
        at = s["rows"][at].long()
    y = torch.bmm(s["X"][at].float(), s["W"][s["active"]].float())
    if s["glu"]:
        gate, up = y.chunk(2, dim=2)
        y = gate / (1.0 + torch.exp(-gate)) * up
    group, place = _places(s["offsets"], n)
    return y[torch.searchsorted(s["active"], group), place].bfloat16()


def _combine(s):
    y = s["Y"][s["slots"].clamp(min=0).long()].float()
    w = torch.where(s["slots"] >= 0, s["weights"], 0.0)
    out = (y * w[:, :, None]).sum(1)
    if s["partials"] is not None:
        out = out + s["partials"].float().sum(0)
    return out.bfloat16()


def _lora(s):
    at = s["rows"][_padded(s["offsets"], s["most"], s["M"])].long()
    h = torch.bmm(s["X"][at].float(), s["down"].float())
    delta = torch.bmm(h, s["up"].float()) * s["scale"][:, None, None]
    out = s["base"].float()
    out[s["rows"][:s["n"]].long()] += delta[_places(s["offsets"], s["n"])]
    return out.bfloat16()


def run(state):
    s = state
    if not own:
        return {"route": _route, "experts": _experts, "combine": _combine, "lora": _lora}[s["op"]](s)
    import tensor_bf16_gemm_amd as gc
    if s["op"] == "route":
        r = gc.moe_route(s["logits"], s["k"], score=s["score"], renormalize=s["renorm"])
        return dict(ids=r.ids, weights=r.weights, offsets=r.offsets, rows=r.rows, slots=r.slots)
    if s["op"] == "experts":
        return gc.grouped_gemm(s["X"], s["W"], s["offsets"], s["rows"],
                               act="silu_glu" if s["glu"] else None)
    if s["op"] == "combine":
        return gc.moe_combine(s["Y"], s["slots"], s["weights"], s["partials"])
    return gc.lora_add(s["base"], s["X"], s["down"], s["up"], s["scale"], s["offsets"], s["rows"])


def work(case):
    c = case
    if c["op"] == "route":
        pairs = c["T"] * c["k"]
        b = c["T"] * c["E"] * (2 if c["dtype"] == "bf16" else 4) + pairs * 16 + (c["E"] + 1) * 4
        return dict(bytes=b, flops=c["T"] * c["E"])
    if c["op"] == "experts":
        rows = c["T"] * c["k"]
        used = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])
        b = 2 * ((c["T"] if c["gather"] else rows) * c["K"] + used * c["K"] * c["N"]
                 + rows * (c["N"] // 2 if c["glu"] else c["N"]))
        return dict(bytes=b + 4 * (c["E"] + rows), flops=2 * rows * c["K"] * c["N"])
    if c["op"] == "combine":
        pairs = c["T"] * c["k"]
        b = 2 * c["N"] * (pairs * c["local"] + (c["peers"] + 1) * c["T"]) + 8 * pairs
        return dict(bytes=b, flops=c["N"] * (2 * pairs * c["local"] + c["peers"] * c["T"]))
    rows = c["M"] * (1.0 - c["none"])
    used = c["G"] * (1.0 - (1.0 - 1.0 / c["G"]) ** rows)
    b = 2 * (rows * c["K"] + 2 * c["M"] * c["N"] + used * c["r"] * (c["K"] + c["N"])) + 4 * c["M"]
    return dict(bytes=b, flops=2 * rows * c["r"] * (c["K"] + c["N"]))


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        x = s["logits"].double()
        out = torch.zeros((s["T"], s["k"]), dtype=torch.float64, device=DEV)
        left = x.clone()
        score = torch.softmax(x, 1) if s["score"] == "softmax" else torch.sigmoid(x)
        for j in range(min(s["k"], s["E"])):      # the next largest, again and again
            best = left.amax(1, keepdim=True)
            at = (left == best).int().argmax(1, keepdim=True)
            out[:, j] = torch.where(best > -math.inf, score.gather(1, at), 0.0)[:, 0]
            left.scatter_(1, at, -math.inf)
        if s["renorm"]:
            out = out / out.sum(1, keepdim=True).clamp(min=1e-300)
        return dict(ids=None, weights=out, offsets=None, rows=None, slots=None)
    if s["op"] == "experts":
        at = s["offsets"].tolist()
        n = s["N"] // 2 if s["glu"] else s["N"]
        out = torch.empty((s["T"] * s["k"], n), dtype=torch.float64, device=DEV)
        for e in range(s["E"]):
            lo, hi = at[e], at[e + 1]
            if lo == hi:
                continue
            x = s["X"][s["rows"][lo:hi].long()] if s["gather"] else s["X"][lo:hi]
            y = x.double() @ s["W"][e].double()
            out[lo:hi] = torch.nn.functional.silu(y[:, :n]) * y[:, n:] if s["glu"] else y
        return out
    if s["op"] == "combine":
        out = torch.zeros((s["T"], s["N"]), dtype=torch.float64, device=DEV)
        for j in range(s["k"]):
            here = torch.nonzero(s["slots"][:, j] >= 0).flatten()
            out[here] += s["weights"][here, j, None].double() * s["Y"][s["slots"][here, j].long()].double()
        for p in range(s["peers"]):
            out += s["partials"][p].double()
        return out
    out = s["base"].double()
    for a in range(s["G"]):
        mine = torch.nonzero(s["ids"] == a).flatten()
        h = s["X"][mine].double() @ s["down"][a].double()
        out[mine] += s["scale"][a].double() * (h @ s["up"][a].double())
    return out
