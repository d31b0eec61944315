"""The routed and grouped operators against plain 64-bit forms (grouped_ref),
at the sizes and masks where they can go wrong."""
import math

import pytest
import torch

import grouped_ref as ref
import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = math.inf
SENTINEL = 0x7FC1


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def filled(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)


def offsets_of(sizes):
    return torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


# ---- router and grouping ----

def check_routing(logits, k, **kw):
    T, E = logits.shape
    bias = kw.get("bias")
    log(f"route T={T} E={E} k={k} {logits.dtype} { {a: b for a, b in kw.items() if a != 'bias'} } bias={bias is not None}")
    r = gc.moe_route(logits.to(DEV), k, **{**kw, **({"bias": bias.to(DEV)} if bias is not None else {})})
    ids, w = ref.route(logits, k, **kw)
    assert torch.equal(r.ids.cpu(), ids)
    # exp and the division: a few units; x - max rounds by |x - max| u; the sum by E u
    finite = torch.where(torch.isfinite(logits.float()), logits.float().abs(), 0.0)
    bound = (2 * float(finite.max()) + E + 32) * 2 * ref.U if T * E else 0.0
    assert torch.all((r.weights.cpu().double() - w).abs() <= bound * w.abs() + 1e-37)
    for got, want, name in zip((r.offsets, r.rows, r.slots), ref.group(ids, E), ("offsets", "rows", "slots")):
        assert torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (1, 8, 8), (1, 3, 5), (7, 63, 3), (64, 64, 8),
                                   (128, 65, 8), (129, 100, 8), (300, 256, 8), (33, 257, 16),
                                   (40, 513, 4), (37, 1024, 2), (1100, 5, 1), (2500, 40, 6)])
@pytest.mark.parametrize("score,renorm,dtype", [("softmax", True, torch.float32),
                                                ("softmax", False, torch.bfloat16),
                                                ("sigmoid", True, torch.bfloat16),
                                                ("sigmoid", False, torch.float32)])
def test_route(T, E, k, score, renorm, dtype):
    logits = (torch.randn((T, E), generator=gen(T + E + k)) * 2).to(dtype)   # bf16: ties among them
    check_routing(logits, k, score=score, renormalize=renorm, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masked_and_infinite(score, renorm):
    E, k = 70, 4
    x = torch.randn((12, E), generator=gen(3))
    x[0] = -INF                                   # nothing left
    x[1] = math.nan
    x[2, 1:] = -INF                               # one left
    x[3, ::2] = math.nan
    x[4] = 0.0
    x[4, ::3] = -0.0                              # equal to +0
    x[5] = torch.finfo(torch.float32).min         # the lowest value is not a mask
    x[6, 10] = INF
    x[7, 10] = x[7, 69] = INF
    x[8] = INF
    x[9] = -INF
    x[9, 69] = torch.finfo(torch.float32).min
    x[10] = 1e-40                                 # subnormal and equal
    if score == "sigmoid":
        x[5], x[9, 69] = -80.0, -80.0             # sigmoid of the lowest value is 0
    check_routing(x, k, score=score, renormalize=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [9, 400])
def test_route_bias(score, T):
    """Selection by score + bias, weights without it.  The biases are further
    apart than any two scores, so that rounding decides no choice."""
    E, k = 48, 5
    g = gen(T)
    x = torch.randn((T, E), generator=g)
    x[T // 2, 3:] = -INF
    bias = 2.0 * torch.randperm(E, generator=g).float()
    check_routing(x, k, score=score, bias=bias, renormalize=True)
    check_routing(x, k, score=score, bias=bias, renormalize=False)


def test_route_strided_rows():
    x = torch.randn((70, 96), generator=gen(5))
    d = x.to(DEV)
    for a, b, s in ((0, 64, 1), (3, 67, 1), (1, 90, 2)):
        r = gc.moe_route(d[::s, a:b], 4)
        assert torch.equal(r.ids.cpu(), ref.route(x[::s, a:b], 4)[0])


@pytest.mark.parametrize("T,k,groups", [(0, 1, 3), (1, 1, 1), (64, 1, 5), (1024, 1, 1024), (1025, 1, 7),
                                        (341, 3, 9), (342, 3, 9), (5000, 1, 33), (20000, 2, 300)])
def test_group_rows(T, k, groups):
    ids = torch.randint(-2, groups + 2, (T, k), generator=gen(T), dtype=torch.int32)
    if T > 4:
        ids[T // 3: T // 2] = groups // 2         # a run of one group
    ids = ids[:, 0].contiguous() if k == 1 else ids
    log(f"group_rows T={T} k={k} groups={groups}")
    for got, want, name in zip(gc.group_rows(ids.to(DEV), groups), ref.group(ids, groups),
                               ("offsets", "rows", "slots")):
        assert torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("T,k,groups", [(2_200_000, 1, 3), (140_000, 16, 1000)])
def test_group_rows_large(T, k, groups):
    """So many items that the blocks grow in number, nearly all of them in one group."""
    ids = torch.randint(0, groups, (T, k), generator=gen(9), dtype=torch.int32)
    ids[torch.rand((T, k), generator=gen(10)) < 0.9] = 1
    key, order = torch.sort(ids.flatten(), stable=True)
    g = gc.group_rows(ids.to(DEV), groups)
    assert torch.equal(g.offsets.cpu(), torch.searchsorted(key, torch.arange(groups + 1, dtype=torch.int32)).int())
    assert torch.equal(g.rows.cpu(), (order // k).int())
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k)
    assert torch.equal(g.slots.cpu().flatten().long(), slots)


# ---- grouped products ----

SIZES = [[1], [0, 0, 5, 0], [16, 17, 0, 33, 1], [64, 65, 1, 63], [130, 0, 257], [7] * 30, [300, 520, 3],
         [1700, 0, 200, 190, 60, 129]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s[:5])))
@pytest.mark.parametrize("K,N", [(8, 16), (32, 48), (40, 272), (256, 128), (904, 336), (2064, 64)])
@pytest.mark.parametrize("act", [None, "silu_glu"])
def test_grouped_gemm(sizes, K, N, act):
    g = gen(K + N + len(sizes))
    S, E, T = sum(sizes), len(sizes), max(1, sum(sizes) // 2)
    W = randn(g, E, K, N, scale=K ** -0.5)
    off = offsets_of(sizes)
    rows = torch.randint(0, T, (S,), generator=g, dtype=torch.int32)
    for X, r in ((randn(g, T, K), rows), (randn(g, S, K), None)):
        want, tol = ref.grouped(X, W, off, r, act)
        for ws in (None, False):
            log(f"grouped_gemm sizes={sizes[:6]} K={K} N={N} act={act} gather={r is not None} ws={ws}")
            got = gc.grouped_gemm(*dev(X, W, off, r), act=act, workspace=ws)
            ref.check(got, want, tol, f"gather={r is not None} ws={ws}")


@pytest.mark.parametrize("rows_per", [3, 40, 200])
def test_grouped_gemm_integers(rows_per):
    """Small integers: every sum is exact in fp32, so any split of K gives the same bits."""
    g = gen(rows_per)
    E, K, N = 5, 1032, 520
    X = torch.randint(-2, 3, (E * rows_per, K), generator=g).bfloat16()
    W = torch.randint(-2, 3, (E, K, N), generator=g).bfloat16()
    off = offsets_of([rows_per] * E)
    want, _ = ref.grouped(X, W, off)
    for ws in (None, False):
        got = gc.grouped_gemm(*dev(X, W, off), workspace=ws)
        assert torch.equal(got.cpu(), want.bfloat16())


RAGGED = [600, 0, 1, 31, 32, 33, 64, 65, 97, 128, 129, 161, 193, 225, 255, 256, 257, 300, 5, 0, 513, 40, 70, 2, 90, 7,
          100, 0, 130, 17]


@pytest.mark.parametrize("sizes,K,N,act,kind", [
    ([1, 0, 5, 16, 2, 0, 9, 17], 1064, 520, None, "stream 16"),
    ([1, 0, 5, 16, 2, 0, 9, 17], 1064, 528, "silu_glu", "stream 16"),
    ([12, 33, 0, 16], 2072, 272, "silu_glu", "stream 32"),
    ([40, 65, 130, 7], 2072, 264, None, "stream 64"),
    (RAGGED, 1064, 2080, None, "tiles"),
    (RAGGED, 1064, 2080, "silu_glu", "tiles"),
    ([2] * 29 + [60], 2056, 2072, None, "tiles"),
    ([2] * 59 + [60], 1064, 2080, None, "tiles"),
    ([130, 0, 270], 4104, 4112, "silu_glu", "split"),
    ([130, 0, 270], 4104, 4112, None, "split"),
    ([700, 500], 7176, 2328, None, "split")])
def test_grouped_gemm_by_plan(sizes, K, N, act, kind):
    """Every way the products are run, over groups of very different sizes."""
    S, E = sum(sizes), len(sizes)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    pl = gc.grouped_plan(S, K, N, E, act=act, cus=cus)
    got = "split" if pl["splits"] > 1 else "tiles" if pl["tiles"] else f"stream {pl['block_rows']}"
    assert got == kind
    g = gen(S + K)
    T = S // 2 + 1
    X, W = randn(g, T, K), randn(g, E, K, N, scale=K ** -0.5)
    rows, off = torch.randint(0, T, (S,), generator=g, dtype=torch.int32), offsets_of(sizes)
    want, tol = ref.grouped(X, W, off, rows, act)
    d = dev(X, W, off, rows)
    for ws in (None, False):
        out = filled(S + 3, want.shape[1])          # (not a row past the last is touched)
        log(f"{kind}: S={S} E={E} K={K} N={N} act={act} ws={ws} {pl}")
        gc.grouped_gemm(*d, act=act, workspace=ws, out=out[:S])
        ref.check(out[:S], want, tol, f"ws={ws}")
        assert torch.all(out[S:].view(torch.int16) == SENTINEL)
        again = gc.grouped_gemm(*d, act=act, workspace=ws)
        assert torch.equal(again, out[:S])


def test_grouped_gemm_many_groups():
    """1024 groups, most of them empty or of one row."""
    g = gen(77)
    E, K, N = 1024, 40, 72
    sizes = torch.randint(0, 4, (E,), generator=g)
    sizes[::3] = 0
    sizes[5], sizes[1023] = 300, 41
    S = int(sizes.sum())
    X, W, off = randn(g, S, K), randn(g, E, K, N), offsets_of(sizes.tolist())
    want, tol = ref.grouped(X, W, off)
    ref.check(gc.grouped_gemm(*dev(X, W, off)), want, tol, "1024 groups")


def test_grouped_gemm_untouched_and_out_of_range():
    """Positions of no group stay as they are; rows outside X read as zeros; offsets outside
    [0, S] are clamped."""
    g = gen(11)
    K, N, T, S = 72, 136, 20, 50
    X, W = randn(g, T, K), randn(g, 4, K, N)
    rows = torch.randint(0, T, (S,), generator=g, dtype=torch.int32)
    rows[7], rows[8], rows[9] = -1, T, 2 ** 31 - 1
    for off in ([3, 10, 10, 30, 41], [0, 60, 60, 90, 1000], [-5, 4, 4, 4, 4], [0, 0, 0, 0, 0],
                [50, 50, 50, 50, 50]):
        off = torch.tensor(off, dtype=torch.int32)
        want, tol = ref.grouped(X, W, off, rows)
        out = filled(S, N)
        log(f"offsets {off.tolist()}")
        gc.grouped_gemm(*dev(X, W, off, rows), out=out)
        ref.check(out, want, tol, str(off.tolist()))
        free = torch.isnan(want)
        assert torch.all(out.cpu().view(torch.int16)[free] == SENTINEL)


def test_grouped_gemm_infinite_stays_in_its_row():
    g = gen(12)
    K, N = 72, 64                                  # K past a whole step: the tail must not mix rows
    X, W = randn(g, 40, K), randn(g, 2, K, N)
    X[5, 3], X[20, K - 1], X[21, 0] = INF, math.nan, -INF
    off = offsets_of([18, 22])
    got = gc.grouped_gemm(*dev(X, W, off)).cpu()
    bad = ~torch.isfinite(got.float()).all(1)
    assert bad.nonzero().flatten().tolist() == [5, 20, 21]


@pytest.mark.parametrize("act", [None, "silu_glu"])
def test_grouped_gemm_empty(act):
    X, W = randn(gen(0), 0, 64).to(DEV), randn(gen(1), 3, 64, 32).to(DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert gc.grouped_gemm(X, W, off, act=act).shape == (0, 16 if act else 32)
    # K = 0: every product is zero
    out = filled(5, 16 if act else 32)
    gc.grouped_gemm(torch.empty((5, 0), dtype=torch.bfloat16, device=DEV),
                    torch.empty((3, 0, 32), dtype=torch.bfloat16, device=DEV),
                    offsets_of([2, 0, 3]).to(DEV), out=out, act=act)
    assert torch.all(out == 0)


def test_grouped_gemm_weights_past_32_bits():
    """The last expert's weights begin 4.3 GB into W."""
    E, K, N = 45, 7168, 6720
    W = torch.zeros((E, K, N), dtype=torch.bfloat16, device=DEV)
    g = gen(7)
    last, X = randn(g, K, N, scale=K ** -0.5), randn(g, 5, K)
    W[E - 1] = last.to(DEV)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = 2
    off[E] = 5
    out = gc.grouped_gemm(X.to(DEV), W, off.to(DEV)).cpu()
    want, tol = ref.grouped(X[2:], last[None], torch.tensor([0, 3], dtype=torch.int32))
    assert torch.all(out[:2] == 0)
    ref.check(out[2:], want, tol, "last expert")


def test_grouped_gemm_same_bits_every_time():
    """A tile cut along K is summed in the order of K, whoever arrives last."""
    g = gen(21)
    X, W = dev(randn(g, 24, 7168), randn(g, 8, 7168, 384, scale=7168 ** -0.5))
    off = offsets_of([3] * 8).to(DEV)
    first = gc.grouped_gemm(X, W, off, act="silu_glu")
    for _ in range(20):
        assert torch.equal(gc.grouped_gemm(X, W, off, act="silu_glu"), first)


# ---- combine ----

@pytest.mark.parametrize("T,k,N,peers", [(1, 1, 8, 0), (3, 2, 520, 1), (17, 8, 1024, 7), (5, 16, 504, 15),
                                         (130, 6, 2056, 3)])
@pytest.mark.parametrize("local", [1.0, 0.4, 0.0])
def test_combine(T, k, N, peers, local):
    g = gen(T + k + N)
    S = T * k + 3
    Y, w = randn(g, S, N), torch.randn((T, k), generator=g)
    slots = torch.randperm(S, generator=g)[:T * k].int().reshape(T, k)
    slots[torch.rand((T, k), generator=g) >= local] = -1
    if T > 1:
        slots[1, 0] = S                            # outside Y: skipped as -1 is
        w[slots < 0] = math.nan                    # the weight of a missing slot is not read
        w[1, 0] = math.nan
    P = randn(g, peers, T, N) if peers else None
    want, tol = ref.combine(Y, slots, w, P)
    log(f"combine T={T} k={k} N={N} peers={peers} local={local}")
    ref.check(gc.moe_combine(*dev(Y, slots, w, P)), want, tol, "combine")


def test_combine_row_slice_of_peers():
    """One rank's rows, as GEMM-RS keeps them: a row slice of slots, weights and every partial."""
    g = gen(2)
    T, k, N, lo, hi = 40, 3, 264, 11, 29
    Y, w, P = randn(g, T * k, N), torch.rand((T, k), generator=g), randn(g, 4, T, N)
    slots = torch.arange(T * k, dtype=torch.int32).reshape(T, k)
    want, tol = ref.combine(Y, slots, w, P)
    d = dev(Y, slots, w, P)
    got = gc.moe_combine(d[0], d[1][lo:hi], d[2][lo:hi], d[3][:, lo:hi])
    ref.check(got, want[lo:hi], tol[lo:hi], "slice")


# ---- adapters ----

@pytest.mark.parametrize("M,K,N,r,G", [(1, 64, 64, 8, 1), (5, 72, 264, 16, 3), (64, 904, 520, 24, 32),
                                       (70, 256, 136, 40, 2), (200, 2056, 328, 64, 3),
                                       (150, 128, 1032, 104, 9), (90, 136, 72, 128, 2), (33, 40, 16, 32, 40)])
@pytest.mark.parametrize("none", [0.0, 0.3, 1.0])
def test_lora_add(M, K, N, r, G, none):
    g = gen(M + K + N + r)
    X, base = randn(g, M, K), randn(g, M, N)
    down, up = randn(g, G, K, r, scale=K ** -0.5), randn(g, G, r, N, scale=r ** -0.5)
    scale = torch.randn(G, generator=g)
    ids = torch.randint(0, G, (M,), generator=g, dtype=torch.int32)
    ids[torch.rand(M, generator=g) < none] = -1
    want, tol = ref.lora(base, X, down, up, scale, ids)
    off, rows, _ = gc.group_rows(ids.to(DEV), G)
    d = dev(base, X, down, up, scale)
    log(f"lora M={M} K={K} N={N} r={r} G={G} none={none}")
    got = gc.lora_add(*d, off, rows)
    ref.check(got, want, tol, "apart")
    assert torch.equal(d[0].cpu(), base)
    same = gc.lora_add(*d, off, rows, out=d[0])
    assert same is d[0] and torch.equal(same, got), "in place"


def test_lora_add_rows_out_of_range():
    """A row number outside the matrix is neither read nor written."""
    g = gen(4)
    M, K, N, r, G = 20, 64, 72, 16, 2
    d = dev(randn(g, M, N), randn(g, M, K), randn(g, G, K, r), randn(g, G, r, N), torch.ones(G))
    rows = torch.arange(M, dtype=torch.int32)
    want = gc.lora_add(*d, offsets_of([9, 11]).to(DEV), rows.to(DEV))
    rows[4], rows[15] = -3, M
    out = filled(M, N)
    gc.lora_add(*d, offsets_of([9, 11]).to(DEV), rows.to(DEV), out=out)
    for m in range(M):
        if m in (4, 15):
            assert torch.all(out[m].view(torch.int16) == SENTINEL)
        else:
            assert torch.equal(out[m], want[m])


# ---- streams and graphs ----

def layer(x, logits, k, W1, W2, partials):
    r = gc.moe_route(logits, k)
    h = gc.grouped_gemm(x, W1, r.offsets, r.rows, act="silu_glu")
    y = gc.grouped_gemm(h, W2, r.offsets)
    return gc.moe_combine(y, r.slots, r.weights, partials)


def layer_inputs(T, seed):
    g = gen(seed)
    E, K, F = 12, 264, 72
    return dev(randn(g, T, K), torch.randn((T, E), generator=g), randn(g, E, K, 2 * F, scale=K ** -0.5),
               randn(g, E, F, K, scale=F ** -0.5), randn(g, 3, T, K))


@pytest.mark.parametrize("T", [1, 60, 300])
def test_layer_on_its_own_streams(T):
    """Two streams at once, each with the workspace of its own."""
    x, lg, W1, W2, P = layer_inputs(T, T)
    want = layer(x, lg, 4, W1, W2, P)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(layer(x, lg, 4, W1, W2, P))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) for a in got)


def test_layer_in_a_graph():
    x, lg, W1, W2, P = layer_inputs(60, 1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer(x, lg, 4, W1, W2, P)                 # the stream's workspace exists before the capture
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = layer(x, lg, 4, W1, W2, P)
    for seed in range(4):
        nx, nl, *_ = layer_inputs(60, 10 + seed)
        x.copy_(nx)
        lg.copy_(nl)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer(x, lg, 4, W1, W2, P))
        torch.cuda.synchronize()
