"""Cases, plain forms and exact values of the operators between and around the
projections of a layer.

Four operators of one tensor-parallel rank, beside the projections and the
routed operators of this package:

  norm   rms_norm: the sum with the residual and the other ranks' partials, its
         RMS norm, in bf16 or in e4m3 with a scale per row and 128 columns
  quant  quantize_fp8: e4m3 with a scale per row and 128 columns (activations)
         or per block of 128 x 128 (weights)
  gemm   gemm_fp8: the product of two such operands, plus the other ranks'
         partials
  moe    moe_layer: router, experts and combine for a few tokens

Hidden sizes 7168 and 6288 / 3648, the 896 = 7168 / 8 columns of one of
eight ranks, and up to 7 peers are the sizes of workloads/; expert counts and
token counts are generic.
"""
import math

import torch

own = False

DEV = "cuda"
FP8_MAX = 448.0
LEAST = 2.0 ** -100             # a block's largest value counts as at least this


def listed():
    return [
        # A decode step of 16 requests: the other ranks' partials of the
        # projection, the residual, the norm and the next projection's input.
        dict(name="norm_decode", op="norm", M=16, N=7168, peers=7, residual=True, fp8=True,
             weight="bf16"),
        # A prefill chunk after a projection that has summed its peers itself.
        dict(name="norm_prefill", op="norm", M=16384, N=7168, peers=0, residual=True, fp8=True,
             weight="bf16"),
        # The input of a projection that no norm precedes, a prefill chunk.
        dict(name="quant_rows", op="quant", M=4096, K=7168, blocks=False),
        # Weights as they are loaded.
        dict(name="quant_weight", op="quant", M=6288, K=7168, blocks=True),
        # One token, one rank's columns: the smallest product, all latency.
        dict(name="gemm_token", op="gemm", M=1, N=7168, K=896, peers=0),
        # A decode batch: the weights' bytes, 7 peers hold partials.
        dict(name="gemm_decode", op="gemm", M=16, N=6288, K=7168, peers=7),
        # A small prefill chunk of the narrower projection.
        dict(name="gemm_chunk", op="gemm", M=256, N=3648, K=7168, peers=7),
        # A ragged batch: no size a multiple of a tile or of a block.
        dict(name="gemm_odd", op="gemm", M=777, N=3640, K=1040, peers=3),
        # The projection of a prefill chunk with its reduction: the largest.
        dict(name="gemm_prefill", op="gemm", M=4096, N=6288, K=7168, peers=7),
        # One token, 8 of 64 experts.
        dict(name="moe_token", op="moe", T=1, E=64, k=8, K=7168, F=896, N=7168, peers=0,
             score="softmax", local=1.0, masked=0.0),
        # Small experts, odd sizes, a few of them out of service, a third of
        # them on this rank.
        dict(name="moe_odd", op="moe", T=5, E=60, k=6, K=1048, F=456, N=1048, peers=2,
             score="sigmoid", local=0.34, masked=0.1),
        # A decode batch of 16 requests, 7 peers hold partials.
        dict(name="moe_decode", op="moe", T=16, E=64, k=8, K=7168, F=896, N=7168, peers=7,
             score="softmax", local=1.0, masked=0.0),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, -(-lo // step) * step), hi // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "gemm", "gemm", "gemm", "moe", "moe"])
    if op == "norm":
        N, peers = _spread(rng, 128, 16384, 16), rng.choice([0, 0, 1, 3, 7])
        most = 16384 * 7168 * 3 // ((peers + 3) * N)
        return dict(op=op, M=_spread(rng, 1, min(16384, most)), N=N, peers=peers,
                    residual=rng.random() < 0.7, fp8=rng.random() < 0.6,
                    weight=rng.choice(["bf16", "f32"]))
    if op == "quant":
        return dict(op=op, M=_spread(rng, 1, 6288), K=_spread(rng, 16, 7168, 16),
                    blocks=rng.random() < 0.4)
    if op == "gemm":
        N, K = _spread(rng, 64, 7168, 8), _spread(rng, 64, 7168, 16)
        return dict(op=op, M=_spread(rng, 1, 4096), N=min(N, 6288), K=K,
                    peers=rng.choice([0, 0, 1, 3, 7]))
    K, F, E = _spread(rng, 256, 7168, 8), _spread(rng, 64, 896, 8), _spread(rng, 4, 64)
    return dict(op=op, T=rng.randint(1, 16), E=E, k=rng.randint(1, min(8, E)), K=K, F=F, N=K,
                peers=rng.choice([0, 1, 7]), score=rng.choice(["softmax", "sigmoid"]),
                local=rng.choice([1.0, 1.0, 0.5]), masked=rng.choice([0.0, 0.0, 0.2]))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    x = torch.randn(shape, generator=g, dtype=dtype, device=DEV)
    return x.mul_(scale) if scale != 1.0 else x


def _activations(g, M, K):
    """Rows of different sizes with a few columns that stand out, as a layer's are."""
    x = _randn(g, M, K, dtype=torch.float32)
    x *= torch.exp(0.5 * _randn(g, M, 1, dtype=torch.float32))
    x *= torch.where(torch.rand((1, K), generator=g, device=DEV) < 0.005, 20.0, 1.0)
    return x.bfloat16()


def _blocks(x, rows):
    """x [M,K] padded with zeros to whole blocks, as [M/rows, rows, K/128, 128]."""
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128, 0, -M % rows))
    return x.reshape(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def _quantize(x, rows):
    """e4m3 values and scales [M/rows, K/128] of x [M,K] (32 or 64 bits)."""
    M, K = x.shape
    b = _blocks(x, rows)
    scales = b.abs().amax((1, 3)).clamp(min=LEAST) / FP8_MAX
    q = b / scales[:, None, :, None]
    q = q.reshape(b.shape[0] * rows, -1)[:M, :K]
    return q, scales


def _scaled(q, scales, rows):
    """The values, in the scales' type, that e4m3 q [M,K] with scales [M/rows, K/128] stands for."""
    M, K = q.shape
    b = _blocks(q.to(scales.dtype), rows) * scales[:, None, :, None]
    return b.reshape(b.shape[0] * rows, -1)[:M, :K]


def _rows_of_16_bytes(scales):
    """The scales with rows that begin on 16 bytes, as quantize_fp8 and rms_norm return them."""
    kb = scales.shape[1]
    return torch.nn.functional.pad(scales, (0, -kb % 4)).contiguous()[:, :kb]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if s["op"] == "norm":
        M, N = s["M"], s["N"]
        s["x"] = _activations(g, M, N)
        s["resid"] = _activations(g, M, N) if s["residual"] else None
        s["partials"] = _randn(g, s["peers"], M, N) if s["peers"] else None
        w = 1.0 + 0.2 * _randn(g, N, dtype=torch.float32)
        s["w"] = w.bfloat16() if s["weight"] == "bf16" else w
    elif s["op"] == "quant":
        s["x"] = (_randn(g, s["M"], s["K"], scale=s["K"] ** -0.5) if s["blocks"]
                  else _activations(g, s["M"], s["K"]))
    elif s["op"] == "gemm":
        M, N, K = s["M"], s["N"], s["K"]
        q, sa = _quantize(_activations(g, M, K).float(), 1)
        s["A"], s["a_scales"] = q.to(torch.float8_e4m3fn), _rows_of_16_bytes(sa)
        q, s["b_scales"] = _quantize(_randn(g, N, K, scale=K ** -0.5).float(), 128)
        s["B"] = q.to(torch.float8_e4m3fn)
        s["partials"] = _randn(g, s["peers"], M, N) if s["peers"] else None
    else:
        T, E, K, F, N = s["T"], s["E"], s["K"], s["F"], s["N"]
        n = max(1, int(E * s["local"]))                 # experts here, from `first` on
        s["first"] = (E - n) // 2
        s["x"] = _randn(g, T, K)
        logits = _randn(g, T, E, dtype=torch.float32)
        if s["masked"] > 0:
            logits = logits.masked_fill(torch.rand((1, E), generator=g, device=DEV) < s["masked"], -math.inf)
            if T > 1:
                logits[T // 2] = -math.inf              # a padding token: no expert at all
        s["logits"] = logits
        s["w1"] = _randn(g, n, K, 2 * F, scale=K ** -0.5)
        s["w2"] = _randn(g, n, F, N, scale=F ** -0.5)
        s["partials"] = _randn(g, s["peers"], T, N) if s["peers"] else None
    return s


def _norm(s):
    h = s["x"].float()
    if s["resid"] is not None:
        h = h + s["resid"].float()
    if s["partials"] is not None:
        h = h + s["partials"].float().sum(0)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["w"].float()
    out = {} if s["resid"] is None and s["partials"] is None else dict(sum=h.bfloat16())
    if not s["fp8"]:
        return dict(out, y=y.bfloat16())
    q, scales = _quantize(y, 1)
    return dict(out, y=q.to(torch.float8_e4m3fn), scales=scales)


def _quant(s):
    q, scales = _quantize(s["x"].float(), 128 if s["blocks"] else 1)
    return dict(q=q.to(torch.float8_e4m3fn), scales=scales)


def _gemm(s):
    out = _scaled(s["A"], s["a_scales"], 1) @ _scaled(s["B"], s["b_scales"], 128).t()
    if s["partials"] is not None:
        out = out + s["partials"].float().sum(0)
    return out.bfloat16()


def _moe(s):
    x, T, E, k = s["logits"], s["T"], s["E"], s["k"]
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    if s["score"] == "softmax":
        high = x.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
        w = torch.exp(top - high) / torch.exp(x - high).sum(1, keepdim=True)
    else:
        w = 1.0 / (1.0 + torch.exp(-top))
    w = torch.where(top > -math.inf, w, 0.0)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0)
    share = torch.zeros((T, E), device=DEV).scatter_(1, ids, w)
    share = share[:, s["first"]:s["first"] + s["w1"].shape[0]].t()     # [experts here, T]
    used = torch.nonzero(share.sum(1)).flatten()
    gate, up = torch.matmul(s["x"].float(), s["w1"][used].float()).chunk(2, dim=2)
    a = (gate / (1.0 + torch.exp(-gate)) * up).bfloat16().float()      # as the experts' products hand it on
    out = (torch.bmm(a, s["w2"][used].float()) * share[used][:, :, None]).sum(0)
    if s["partials"] is not None:
        out = out + s["partials"].float().sum(0)
    return out.bfloat16()


def run(state):
    s = state
    if not own:
        return {"norm": _norm, "quant": _quant, "gemm": _gemm, "moe": _moe}[s["op"]](s)
    import tensor_bf16_gemm_amd as gc
    if s["op"] == "norm":
        r = gc.rms_norm(s["x"], s["w"], residual=s["resid"], partials=s["partials"], eps=1e-6, fp8=s["fp8"])
        return {n: t for n, t in r._asdict().items() if t is not None}
    if s["op"] == "quant":
        return gc.quantize_fp8(s["x"], block_rows=128 if s["blocks"] else 1)._asdict()
    if s["op"] == "gemm":
        return gc.gemm_fp8(s["A"], s["a_scales"], s["B"], s["b_scales"], s["partials"])
    return gc.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], s["k"], first=s["first"], score=s["score"],
                        partials=s["partials"])


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["N"]
        summed = c["residual"] or c["peers"] > 0
        b = n * (2 * (1 + c["residual"] + c["peers"] + summed) + (1 if c["fp8"] else 2))
        if c["fp8"]:
            b += c["M"] * -(-c["N"] // 128) * 4
        return dict(bytes=b + c["N"] * (2 if c["weight"] == "bf16" else 4), flops=6 * n)
    if c["op"] == "quant":
        n = c["M"] * c["K"]
        rows = -(-c["M"] // 128) if c["blocks"] else c["M"]
        return dict(bytes=3 * n + rows * -(-c["K"] // 128) * 4, flops=3 * n)
    if c["op"] == "gemm":
        M, N, K, kb = c["M"], c["N"], c["K"], -(-c["K"] // 128)
        b = M * K + N * K + 4 * kb * (M + -(-N // 128)) + 2 * M * N * (c["peers"] + 1)
        return dict(bytes=b, flops=2 * M * N * K)
    n, up, down = max(1, int(c["E"] * c["local"])), 2 * c["K"] * c["F"], c["F"] * c["N"]
    left = max(c["k"], c["E"] * (1.0 - c["masked"]))     # experts that can be chosen
    tokens = c["T"] - (1 if c["masked"] > 0 and c["T"] > 1 else 0)
    used = n * left / c["E"] * (1.0 - (1.0 - c["k"] / left) ** tokens)
    b = 2 * used * (up + down) + 2 * c["T"] * (c["K"] + (c["peers"] + 1) * c["N"]) + 4 * c["T"] * c["E"]
    return dict(bytes=b, flops=2 * tokens * c["k"] * n / c["E"] * (up + down))


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "norm":
        h = torch.stack([t.to(f64) for t in (s["x"], s["resid"]) if t is not None]).sum(0)
        for p in range(s["peers"]):
            h += s["partials"][p].to(f64)
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / s["N"] + 1e-6) * s["w"].to(f64)
        out = dict(sum=h) if s["residual"] or s["peers"] else {}
        if not s["fp8"]:
            return dict(out, y=y)
        return dict(out, **_exact_codes(y, "y"))
    if s["op"] == "quant":
        if not s["blocks"]:
            return _exact_codes(s["x"].to(f64), "q")
        x, M, K = s["x"].to(f64), s["M"], s["K"]
        scales = torch.empty((-(-M // 128), -(-K // 128)), dtype=f64, device=DEV)
        q = torch.empty_like(x)
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                part = x[128 * i:128 * i + 128, 128 * j:128 * j + 128]
                scales[i, j] = torch.clamp(part.abs().max(), min=LEAST) / FP8_MAX
                q[128 * i:128 * i + 128, 128 * j:128 * j + 128] = _e4m3(part / scales[i, j])
        return dict(q=q, scales=scales)
    if s["op"] == "gemm":
        out = torch.zeros((s["M"], s["N"]), dtype=f64, device=DEV)
        sb = s["b_scales"].to(f64).repeat_interleave(128, 0)[:s["N"]]
        for j in range(sb.shape[1]):
            at = slice(128 * j, min(128 * j + 128, s["K"]))
            a = s["A"][:, at].to(f64) * s["a_scales"][:, j, None].to(f64)
            out += a @ (s["B"][:, at].to(f64) * sb[:, j, None]).t()
        for p in range(s["peers"]):
            out += s["partials"][p].to(f64)
        return out
    x = s["logits"].to(f64)
    score = torch.softmax(x, 1) if s["score"] == "softmax" else torch.sigmoid(x)
    out = torch.zeros((s["T"], s["N"]), dtype=f64, device=DEV)
    if s["partials"] is not None:
        out += s["partials"].to(f64).sum(0)
    for t in range(s["T"]):
        left, chosen = x[t].tolist(), []
        for _ in range(s["k"]):                          # the next largest, again and again
            best = max(left)
            if best == -math.inf:
                break
            chosen.append(left.index(best))
            left[chosen[-1]] = -math.inf
        total = sum(float(score[t, e]) for e in chosen)
        for e in chosen:
            i = e - s["first"]
            if 0 <= i < s["w1"].shape[0]:
                y = s["x"][t].to(f64) @ s["w1"][i].to(f64)
                a = torch.nn.functional.silu(y[:s["F"]]) * y[s["F"]:]
                out[t] += float(score[t, e]) / total * (a @ s["w2"][i].to(f64))
    return out


def _e4m3(v):
    """v (64 bits, |v| at most 448) rounded to the nearest of the values of e4m3, ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    e = torch.where(v.abs() >= torch.exp2(e + 1), e + 1, torch.where(v.abs() < torch.exp2(e), e - 1, e)).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_codes(y, name):
    M, N = y.shape
    scales = torch.empty((M, -(-N // 128)), dtype=torch.float64, device=DEV)
    q = torch.empty_like(y)
    for j in range(scales.shape[1]):
        part = y[:, 128 * j:128 * j + 128]
        scales[:, j] = part.abs().amax(1).clamp(min=LEAST) / FP8_MAX
        q[:, 128 * j:128 * j + 128] = _e4m3(part / scales[:, j, None])
    return {name: q, "scales": scales}
