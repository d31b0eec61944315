"""The operators between and around the projections against plain 64-bit forms
(layer_ref), at the sizes and values where they can go wrong."""
import math

import pytest
import torch

import layer_ref as ref
import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = math.inf, math.nan
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SENTINEL = 0x7FC1


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def filled(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device=DEV).view(BF16)


# ---- norm ----

def rows_of(g, M, N):
    """Rows of very different sizes."""
    return (torch.randn((M, N), generator=g) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g))).bfloat16()


@pytest.mark.parametrize("M,N", [(1, 8), (1, 16), (3, 128), (5, 136), (2, 512), (9, 520), (7, 1024), (33, 1040),
                                 (4, 2048), (700, 2064), (1, 4096), (600, 4112), (513, 7168), (16, 7168), (2, 8192),
                                 (3, 8200), (2, 16384), (1, 16400), (2, 32768), (1030, 64)])
@pytest.mark.parametrize("form", ["bf16", "sum", "fp8", "fp8 sum"])
def test_rms_norm(M, N, form):
    fp8, whole = "fp8" in form, "sum" in form
    if fp8 and N % 16:
        pytest.skip("codes in whole 16-byte rows")
    g = gen(M + N)
    peers = (M + N // 8) % 4 if whole else 0
    x, residual = rows_of(g, M, N), rows_of(g, M, N) if whole else None
    partials = torch.stack([rows_of(g, M, N) for _ in range(peers)]) if peers else None
    w = 1.0 + 0.3 * torch.randn(N, generator=g)
    w = w if N % 32 == 0 else w.bfloat16()
    log(f"rms_norm M={M} N={N} {form} peers={peers} {w.dtype}")
    xd, rd, pd, wd = dev(x, residual, partials, w)
    r = gc.rms_norm(xd, wd, residual=rd, partials=pd, eps=1e-5, fp8=fp8)
    h, dh, y, dy = ref.rms(x, w, residual, partials, 1e-5)
    if whole:
        ref.check(r.sum, h, dh + ref.BF * (h.abs() + dh) + ref.TINY, "sum")
    else:
        assert r.sum is None
    if fp8:
        assert r.scales.shape == (M, -(-N // 128)) and r.y.dtype == E4M3
        ref.check_codes(r.y, r.scales, y, dy, 1, "norm")
    else:
        assert r.scales is None
        ref.check(r.y, y, dy + ref.BF * (y.abs() + dy) + ref.TINY, "y")


def test_rms_norm_in_place():
    """The sum over its own residual (or x), the output over x: as with outputs of their own."""
    g = gen(7)
    x, res, w = dev(randn(g, 37, 1024), randn(g, 37, 1024), randn(g, 1024))
    want = gc.rms_norm(x, w, residual=res)
    a, b = x.clone(), res.clone()
    got = gc.rms_norm(a, w, residual=b, out=a, sum_out=b)
    assert got.y is a and got.sum is b
    assert torch.equal(a, want.y) and torch.equal(b, want.sum)
    a = x.clone()
    got = gc.rms_norm(a, w, residual=res, sum_out=a, fp8=True)
    again = gc.rms_norm(x, w, residual=res, fp8=True)
    assert torch.equal(a, want.sum)
    assert torch.equal(got.y.view(torch.uint8), again.y.view(torch.uint8)) and torch.equal(got.scales, again.scales)


def test_rms_norm_of_a_slice_of_the_peers():
    """The rows of one rank out of larger partials."""
    g = gen(8)
    x, w, p = dev(randn(g, 10, 256), randn(g, 256), randn(g, 5, 40, 256))
    got = gc.rms_norm(x, w, partials=p[:, 20:30])
    want = gc.rms_norm(x, w, partials=p[:, 20:30].contiguous())
    assert torch.equal(got.y, want.y) and torch.equal(got.sum, want.sum)


@pytest.mark.parametrize("N", [256, 1040, 7168])
def test_rms_norm_values_that_are_not_finite(N):
    """A NaN or an infinity stays in its row."""
    x = randn(gen(9), 6, N)
    x[1, 5], x[3, N - 1], x[4] = NAN, INF, 0.0
    w = torch.ones(N)
    y = gc.rms_norm(*dev(x, w)).y.cpu()
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[3, N - 1]) and (y[3, :N - 1] == 0).all()       # inf / inf, x / inf
    assert (y[4] == 0).all()
    rows = [0, 2, 5]
    alone = gc.rms_norm(*dev(x[rows], w)).y.cpu()
    assert torch.equal(y[rows], alone)
    r = gc.rms_norm(*dev(x, w), fp8=True)
    q, s = r.y.float().cpu(), r.scales.cpu()
    assert torch.isnan(q[1]).all() and torch.isnan(s[1]).all()
    assert torch.isnan(q[3, (N - 1) // 128 * 128:]).all() and torch.isnan(s[3, -1]) and (q[3, :128] == 0).all()
    assert (q[4] == 0).all() and torch.isfinite(s[4]).all()


def test_rms_norm_zero_eps_and_empty():
    x = torch.zeros((2, 64), dtype=BF16, device=DEV)
    assert torch.isnan(gc.rms_norm(x, torch.ones(64, device=DEV), eps=0.0).y).all()     # 0 / 0, as the formula
    r = gc.rms_norm(x[:0], torch.ones(64, device=DEV), fp8=True)
    assert r.y.shape == (0, 64) and r.scales.shape == (0, 1)


# ---- quantisation ----

@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (130, 7168), (257, 400), (128, 128), (640, 1040),
                                 (5, 16384)])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize(M, K, rows):
    x = rows_of(gen(M * K), M, K)
    log(f"quantize M={M} K={K} rows={rows}")
    q, s = gc.quantize_fp8(x.to(DEV), block_rows=rows)
    assert s.shape == (-(-M // rows), -(-K // 128))
    y = x.double()
    ref.check_codes(q, s, y, torch.zeros_like(y), rows, "quantize")


def test_quantize_is_exact_where_it_can_be():
    """Values that are a code times a power of two, with 448 of them in every block, come back
    whole; so do zeros, and blocks of subnormals are rounded, not lost."""
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3).float()
    codes = codes[torch.isfinite(codes)]                                  # every finite code
    x = torch.zeros((3, 256))
    x[0, :codes.numel()] = codes * 2.0 ** 20
    x[0, 128] = 448 * 2.0 ** 20
    x[1, :codes.numel()] = codes * 2.0 ** -30
    x[1, 0], x[1, 128] = 448 * 2.0 ** -30, 448 * 2.0 ** -30
    x[2, 3] = 2.0 ** -130
    q, s = gc.quantize_fp8(x.bfloat16().to(DEV))
    back = q.float().cpu() * ref.spread(s.cpu(), 1, 3, 256)
    assert torch.equal(back[:2], x[:2])
    assert torch.equal(s[2].cpu(), torch.full((2,), 2.0 ** -100 / 448)) and (back[2] == 0).all()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("power", [0, 100, 119, -80])
def test_quantize_ties_go_to_the_even_code(rows, power):
    """Halfway between two codes exactly: the even one, at any size of the block's largest value."""
    x = torch.zeros((rows, 128))
    x[0, 0] = 448.0                                       # scale 1 (times the power of two)
    mid = torch.tensor([17.0, 19.0, 21.0, 23.0, 25.0, 27.0, 29.0, 31.0])      # codes are 16, 18, .. 32 here
    want = torch.tensor([16.0, 20.0, 20.0, 24.0, 24.0, 28.0, 28.0, 32.0])
    x[0, 8:16], x[0, 16:24] = mid, -mid
    top = torch.tensor([448.0 * 3 / 4])                   # 336: quotients 4/3 of the values
    x2 = torch.zeros((rows, 128))
    x2[0, 0], x2[0, 8:16] = float(top), mid * 3 / 4
    for v in (x, x2):
        q, s = gc.quantize_fp8((v * 2.0 ** power).bfloat16().to(DEV), block_rows=rows)
        assert torch.equal(q[0, 8:16].float().cpu(), want) and float(q[0, 0]) == 448.0
    q, s = gc.quantize_fp8((x * 2.0 ** power).bfloat16().to(DEV), block_rows=rows)
    assert torch.equal(q[0, 16:24].float().cpu(), -want) and float(s[0, 0]) == 2.0 ** power


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_quantize_values_that_are_not_finite(rows, bad):
    """All of a block that holds one is NaN, the other blocks are as without it."""
    x = randn(gen(3), 200, 400)
    want, ws = gc.quantize_fp8(x.to(DEV), block_rows=rows)
    x[140, 130] = bad
    q, s = gc.quantize_fp8(x.to(DEV), block_rows=rows)
    lo, hi = (140, 141) if rows == 1 else (128, 200)
    block = torch.zeros((200, 400), dtype=torch.bool, device=DEV)
    block[lo:hi, 128:256] = True
    assert torch.isnan(q.float()[block]).all() and torch.isnan(s[140 // rows, 1])
    assert torch.equal(q.view(torch.uint8)[~block], want.view(torch.uint8)[~block])
    rest = torch.ones_like(s, dtype=torch.bool)
    rest[140 // rows, 1] = False
    assert torch.equal(s[rest], ws[rest])


# ---- e4m3 products ----

def operands(M, N, K, seed, peers=0):
    g = gen(seed)
    a, b = rows_of(g, M, K), randn(g, N, K, scale=max(K, 1) ** -0.5)
    A, sa = gc.quantize_fp8(a.to(DEV))
    B, sb = gc.quantize_fp8(b.to(DEV), block_rows=128)
    p = randn(g, peers, M, N) if peers else None
    return A, sa, B, sb, None if p is None else p.to(DEV)


def check_gemm(ops, **kw):
    A, sa, B, sb, p = ops
    got = gc.gemm_fp8(A, sa, B, sb, p, **kw)
    want = ref.gemm(A.float().cpu(), sa.cpu(), B.float().cpu(), sb.cpu(), None if p is None else p.cpu())
    ref.check(got, *want, f"gemm_fp8 {tuple(A.shape)} {B.shape[0]} peers {0 if p is None else p.shape[0]}")
    return got


SIZES = [(1, 8, 16), (1, 16, 128), (1, 136, 7168), (16, 64, 896), (17, 40, 144), (32, 296, 2064), (33, 520, 272),
         (64, 1000, 1040), (65, 264, 400), (100, 256, 128), (128, 512, 1024), (200, 776, 528), (257, 1288, 1296),
         (480, 248, 2048), (513, 264, 16), (1000, 1048, 656)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("peers", [0, 3])
def test_gemm(M, N, K, peers):
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers} plan {gc.gemm_fp8_plan(M, N, K, peers)}")
    ops = operands(M, N, K, M + N + K, peers)
    got = check_gemm(ops)
    again = gc.gemm_fp8(*ops)
    assert torch.equal(got, again)
    check_gemm(ops, workspace=False)


# One size at least for every kind of tile: (rows, columns) of the tile, cut in K or not.
WAYS = [((16, 16), False, 20, 72, 400), ((16, 32), False, 20, 2056, 656), ((32, 16), False, 450, 264, 656),
        ((32, 32), False, 40, 3208, 400), ((32, 64), False, 100, 2056, 1040), ((64, 32), False, 4099, 72, 272),
        ((64, 256), False, 500, 4104, 656), ((128, 256), False, 1800, 2056, 1424), ((128, 256), True, 500, 4104, 4112),
        ((224, 256), False, 2000, 4104, 400), ((224, 256), False, 1990, 4104, 2192), ((224, 256), True, 1800, 2056, 4112),
        ((256, 256), False, 2040, 6664, 656), ((256, 256), False, 2047, 6664, 1936)]


@pytest.mark.parametrize("tile,cut,M,N,K", WAYS)
@pytest.mark.parametrize("peers", [0, 1, 9])
def test_gemm_every_way(tile, cut, M, N, K, peers):
    """Every kind of tile, with rows, columns and K that end inside one, with more blocks of the
    peers than steps of K and with fewer (64-bit values on the GPU)."""
    pl = gc.gemm_fp8_plan(M, N, K, peers)
    log(f"gemm_fp8 M={M} N={N} K={K} peers={peers} plan {pl}")
    A, sa, B, sb, p = operands(M, N, K, M + K, peers)
    want = [t.cpu() for t in ref.gemm(A, sa, B, sb, p)]
    buf = filled(M + 1, N)
    got = gc.gemm_fp8(A, sa, B, sb, p, out=buf[:M])
    ref.check(got, *want, f"{pl}")
    assert (buf.view(torch.int16)[M] == SENTINEL).all()
    assert torch.equal(gc.gemm_fp8(A, sa, B, sb, p), got)


def test_the_ways_are_taken():
    """Each size above is run the way it is there for, with or without peers, on 256 compute units."""
    for tile, cut, M, N, K in WAYS:
        found = [gc.gemm_fp8_plan(M, N, K, p) for p in (0, 1, 9)]
        assert any((f["tile_rows"], f["tile_cols"]) == tile and (f["splits"] > 1) == cut for f in found), (tile, found)


@pytest.mark.parametrize("M", [3, 70, 300])
@pytest.mark.parametrize("form", ["columns first", "odd rows", "one for all", "slice"])
def test_gemm_scales_of_any_strides(M, form):
    N, K = 264, 1168
    A, sa, B, sb, _ = operands(M, N, K, 5)
    if form == "columns first":
        s = sa.t().contiguous().t()
    elif form == "odd rows":
        s = torch.full((M, 13), NAN, device=DEV)[:, 1:11]
        s.copy_(sa)
    elif form == "one for all":
        sa = sa[:1].expand(M, -1).contiguous()
        s = sa[:1].expand(M, -1)
    else:
        wide = torch.full((M, 40), NAN, device=DEV)
        s = wide[:, ::4]
        s.copy_(sa)
    assert torch.equal(gc.gemm_fp8(A, s, B, sb), gc.gemm_fp8(A, sa, B, sb))


@pytest.mark.parametrize("M", [5, 80, 300])
def test_gemm_not_finite_stays_in_its_row_or_column(M):
    N, K = 264, 400
    A, sa, B, sb, _ = operands(M, N, K, 6)
    want = gc.gemm_fp8(A, sa, B, sb)
    nan = torch.tensor([0x7F], dtype=torch.uint8, device=DEV).view(E4M3)
    a, b, s = A.clone(), B.clone(), sa.clone()
    a.view(torch.uint8)[M // 2, 399] = nan.view(torch.uint8)
    s[1, 0] = INF
    got = gc.gemm_fp8(a, s, b, sb)
    rows = [m for m in range(M) if m not in (M // 2, 1)]
    assert torch.isnan(got[M // 2]).all() and not torch.isfinite(got[1]).any()
    assert torch.equal(got[rows], want[rows])
    b.view(torch.uint8)[17, 0] = 0xFF
    got = gc.gemm_fp8(A, sa, b, sb)
    cols = [n for n in range(N) if n != 17]
    assert torch.isnan(got[:, 17]).all() and torch.equal(got[:, cols], want[:, cols])


@pytest.mark.parametrize("M", [7, 90, 300])
def test_gemm_writes_its_rows_only(M):
    """Rows behind the last one, and everything after an output of odd size, stay as they were."""
    N, K = 1032, 656
    A, sa, B, sb, p = operands(M, N, K, 11, 2)
    buf = filled(M + 3, N)
    got = gc.gemm_fp8(A, sa, B, sb, p, out=buf[1:M + 1])
    assert torch.equal(got, gc.gemm_fp8(A, sa, B, sb, p))
    keep = buf.view(torch.int16)
    assert (keep[0] == SENTINEL).all() and (keep[M + 1:] == SENTINEL).all()


@pytest.mark.parametrize("M", [4, 100, 700])
def test_gemm_of_no_columns(M):
    """K = 0: the peers' sum, whichever way the sizes are run."""
    p = randn(gen(M), 5, M, 2056).to(DEV)
    none = lambda n: torch.empty((n, 0), dtype=E4M3, device=DEV)  # noqa: E731
    got = gc.gemm_fp8(none(M), torch.empty((M, 0), device=DEV), none(2056), torch.empty((17, 0), device=DEV), p)
    ref.check(got, *ref.combine_peers(p.cpu()), "peers alone")


def test_gemm_of_nothing():
    A, sa, B, sb, p = operands(4, 16, 32, 1, 2)
    assert gc.gemm_fp8(A[:0], sa[:0], B, sb).shape == (0, 16)
    assert gc.gemm_fp8(A, sa, B[:0], sb[:0]).shape == (4, 0)
    none = torch.empty((4, 0), dtype=E4M3, device=DEV)
    got = gc.gemm_fp8(none, torch.empty((4, 0), device=DEV), torch.empty((16, 0), dtype=E4M3, device=DEV),
                      torch.empty((1, 0), device=DEV), p)
    assert torch.equal(got, p.float().sum(0).bfloat16())


def test_gemm_integers_are_exact():
    """Small whole numbers with scales of one: every sum is exact, so is every output."""
    g = gen(2)
    for M, N, K in ((3, 72, 4096), (70, 264, 1040), (300, 520, 656)):
        a = torch.randint(-2, 3, (M, K), generator=g).float()
        b = torch.randint(-2, 3, (N, K), generator=g).float()
        one = torch.ones((M, -(-K // 128)), device=DEV)
        got = gc.gemm_fp8(a.to(E4M3).to(DEV), one, b.to(E4M3).to(DEV), torch.ones((-(-N // 128), -(-K // 128)), device=DEV))
        assert torch.equal(got.cpu(), (a @ b.t()).bfloat16())


# ---- a layer of experts for a few tokens ----

def layer_inputs(T, E, k, K, F, N, seed, local=None, peers=0, dtype=F32, apart=True):
    g = gen(seed)
    n = local or E
    x = randn(g, T, K)
    # logits far enough apart that rounding decides no choice (bf16: ties are decided by index)
    logits = (torch.randn((T, E), generator=g) * 2).to(dtype)
    w1, w2 = randn(g, n, K, 2 * F, scale=max(K, 1) ** -0.5), randn(g, n, F, N, scale=max(F, 1) ** -0.5)
    return x, logits, w1, w2, randn(g, peers, T, N) if peers else None


def check_layer(ins, k, **kw):
    x, logits, w1, w2, p = ins
    bias = kw.get("bias")
    got = gc.moe_layer(*dev(x, logits, w1, w2), k, partials=None if p is None else p.to(DEV),
                       **{**kw, **({} if bias is None else {"bias": bias.to(DEV)})})
    ref.check(got, *ref.layer(x, logits, w1, w2, k, partials=p, **kw), f"moe_layer {tuple(x.shape)} k {k}")
    return got


@pytest.mark.parametrize("T,E,k,K,F,N", [(1, 1, 1, 8, 8, 8), (1, 8, 2, 64, 40, 72), (1, 64, 8, 1024, 96, 1024),
                                         (2, 3, 5, 40, 24, 136), (5, 60, 6, 1048, 456, 264), (16, 64, 8, 264, 72, 520),
                                         (15, 16, 4, 520, 128, 128), (16, 64, 8, 256, 136, 384),
                                         (16, 100, 16, 72, 64, 64), (9, 300, 8, 136, 48, 200),
                                         (3, 1024, 16, 64, 32, 64), (13, 7, 7, 2048, 320, 1032)])
@pytest.mark.parametrize("score,dtype,peers", [("softmax", F32, 0), ("sigmoid", BF16, 3)])
def test_layer(T, E, k, K, F, N, score, dtype, peers):
    log(f"moe_layer T={T} E={E} k={k} K={K} F={F} N={N} {score} {dtype} peers={peers}")
    ins = layer_inputs(T, E, k, K, F, N, T + E + K, peers=peers, dtype=dtype)
    got = check_layer(ins, k, score=score, renormalize=peers == 0, scale=1.5)
    again = gc.moe_layer(*dev(*ins[:4]), k, partials=None if ins[4] is None else ins[4].to(DEV), score=score,
                         renormalize=peers == 0, scale=1.5)
    assert torch.equal(got, again)


@pytest.mark.parametrize("T,first,local", [(1, 0, 3), (6, 5, 4), (16, 9, 3), (4, 11, 1)])
def test_layer_of_a_part_of_the_experts(T, first, local):
    check_layer(layer_inputs(T, 12, 3, 136, 72, 264, T, local=local, peers=2), 3, first=first)


def test_layer_biased():
    ins = layer_inputs(8, 24, 4, 64, 32, 64, 5)
    check_layer(ins, 4, score="sigmoid", bias=2.0 * torch.randperm(24, generator=gen(1)).float())


@pytest.mark.parametrize("peers", [0, 2])
def test_layer_tokens_without_an_expert(peers):
    """Rows whose logits leave nothing get the peers' sum alone, and so do all rows where no chosen
    expert is here."""
    ins = layer_inputs(6, 10, 2, 64, 40, 136, 8, peers=peers)
    ins[1][2] = -INF
    ins[1][4] = NAN
    ins[1][5, 1:] = -INF
    got = check_layer(ins, 2)
    alone = ins[4].float().sum(0).bfloat16() if peers else torch.zeros((6, 136), dtype=BF16)
    assert torch.equal(got[[2, 4]].cpu(), alone[[2, 4]])
    x, logits, w1, w2, p = ins
    logits[:, 6:] = -INF
    none = gc.moe_layer(*dev(x, logits, w1[:4], w2[:4]), 2, first=6, partials=None if p is None else p.to(DEV))
    assert torch.equal(none.cpu(), alone)


def test_layer_other_rows_are_not_touched():
    """Infinities and NaN in an expert's weights, or in a token, reach the rows that chose it alone."""
    x, logits, w1, w2, _ = layer_inputs(8, 6, 2, 72, 40, 136, 12)
    want = gc.moe_layer(*dev(x, logits, w1, w2), 2)
    ids, _ = ref.g.route(logits, 2)
    hit = (ids == 3).any(1)
    assert 0 < int(hit.sum()) < 8
    b1, b2 = w1.clone(), w2.clone()
    b1[3], b2[3] = INF, NAN
    for a, b in ((b1, w2), (w1, b2)):
        got = gc.moe_layer(*dev(x, logits, a, b), 2)
        assert torch.equal(got[~hit], want[~hit]) and torch.isnan(got[hit]).all()
    y = x.clone()
    y[5, 3] = NAN
    got = gc.moe_layer(*dev(y, logits, w1, w2), 2)
    rows = [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(got[rows], want[rows]) and torch.isnan(got[5]).all()


def test_layer_is_the_routed_operators_together():
    """The same choice and activations as moe_route and grouped_gemm."""
    x, logits, w1, w2, p = dev(*layer_inputs(12, 32, 4, 264, 72, 520, 3, peers=2))
    r = gc.moe_route(logits, 4)
    a = gc.grouped_gemm(x, w1, r.offsets, r.rows, act="silu_glu")
    y = gc.grouped_gemm(a, w2, r.offsets)
    want = gc.moe_combine(y, r.slots, r.weights, p)
    got = gc.moe_layer(x, logits, w1, w2, 4, partials=p)
    # the chain rounds every expert's output, the layer only the sum
    e = gc.moe_combine(y.abs(), r.slots, r.weights, p.abs()).double()
    assert torch.all((got.double() - want.double()).abs() <= 3 * ref.BF * e)


def test_layer_of_nothing():
    x, logits, w1, w2, p = dev(*layer_inputs(3, 4, 2, 16, 8, 24, 3, peers=1))
    assert gc.moe_layer(x[:0], logits[:0], w1, w2, 2).shape == (0, 24)
    got = gc.moe_layer(x, logits, w1[:, :, :0].contiguous(), w2[:, :0].contiguous(), 2, partials=p)
    assert torch.equal(got, p[0])
    got = gc.moe_layer(x[:, :0].contiguous(), logits, w1[:, :0].contiguous(), w2, 2)
    assert (got == 0).all()


# ---- all of them, as a layer uses them ----

@pytest.mark.parametrize("T", [1, 13, 16])
def test_a_layer(T):
    """The residual stream of one rank through norm, e4m3 projection with its peers, norm, experts
    with their peers, eagerly and as a captured graph that is replayed with other inputs."""
    hidden, inner, experts, k, ranks = 1024, 136, 24, 4, 4
    g = gen(T)
    x, wn1, wn2 = dev(randn(g, T, hidden), 1 + randn(g, hidden, scale=0.1), 1 + randn(g, hidden, scale=0.1))
    wq, wqs = gc.quantize_fp8(randn(g, hidden, hidden, scale=hidden ** -0.5).to(DEV), block_rows=128)
    router = randn(g, hidden, experts, scale=hidden ** -0.5).to(DEV)
    w1, w2 = dev(randn(g, experts, hidden, 2 * inner, scale=hidden ** -0.5),
                 randn(g, experts, inner, hidden, scale=inner ** -0.5))
    pp, mp = dev(randn(g, ranks - 1, T, hidden), randn(g, ranks - 1, T, hidden))

    def step():
        n1 = gc.rms_norm(x, wn1, fp8=True)
        o = gc.gemm_fp8(n1.y, n1.scales, wq, wqs, pp)
        n2 = gc.rms_norm(o, wn2, residual=x)
        logits = (n2.y.float() @ router.float())
        y = gc.moe_layer(n2.y, logits, w1, w2, k, partials=mp)
        return n1, o, n2, logits, y, gc.rms_norm(y, wn1, residual=n2.sum)

    n1, o, n2, logits, y, last = step()
    c = lambda t: t.cpu()  # noqa: E731
    ref.check_codes(n1.y, n1.scales, *ref.rms(c(x), c(wn1))[2:], 1, "first norm")
    ref.check(o, *ref.gemm(n1.y.float().cpu(), c(n1.scales), wq.float().cpu(), c(wqs), c(pp)), "projection")
    h, dh, v, dv = ref.rms(c(o), c(wn2), c(x))
    ref.check(n2.y, v, dv + ref.BF * (v.abs() + dv) + ref.TINY, "second norm")
    ref.check(y, *ref.layer(c(n2.y), c(logits), c(w1), c(w2), k, partials=c(mp)), "experts")
    h, dh, v, dv = ref.rms(c(y), c(wn1), c(n2.sum))
    ref.check(last.sum, h, dh + ref.BF * (h.abs() + dh) + ref.TINY, "residual")

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
        for seed in range(4):
            x.copy_(randn(gen(100 + seed), T, hidden))
            pp.copy_(randn(gen(200 + seed), ranks - 1, T, hidden))
            graph.replay()
            torch.cuda.synchronize()
            want = step()
            torch.cuda.synchronize()
            for a, b in zip((out[1], out[4], out[5].y, out[5].sum), (want[1], want[4], want[5].y, want[5].sum)):
                assert torch.equal(a, b), seed


# ---- offsets past 32 bits, outputs in larger buffers, refusals ----

@pytest.mark.parametrize("values", ["any bits", "normal"])
def test_rms_norm_past_four_gigabytes(values):
    """(Of any bits, the squares' sums overflow and the codes are NaN: bits are compared,
    with as many rows as take the same kernel, whose sums have the same order.)"""
    M, N = 290_000, 8192                                  # 4.75 GB
    x = torch.empty((M, N), dtype=BF16, device=DEV)
    if values == "normal":
        x.normal_()
    else:
        x.view(torch.int16).random_(-16000, 16000)
    w = torch.ones(N, device=DEV)
    rows = torch.tensor([0, 131_071, 262_143, 262_144, M - 1], device=DEV)
    few, bits = x[rows].repeat(128, 1), {E4M3: torch.uint8, F32: torch.int32, BF16: torch.int16}
    for got, want in ((gc.rms_norm(x, w, residual=x, fp8=True), gc.rms_norm(few, w, residual=few, fp8=True)),
                      (gc.quantize_fp8(x), gc.quantize_fp8(few))):
        for a, b in zip(got, want):
            assert torch.equal(a.view(bits[a.dtype])[rows] if a.dtype != F32 else a[rows].view(torch.int32),
                               b.contiguous().view(bits[b.dtype])[:5])


def test_layer_weights_past_four_gigabytes():
    T, E, K, F = 3, 130, 4096, 2048                       # w1 4.4 GB
    x, logits = randn(gen(1), T, K), torch.zeros((T, E))
    logits[0, 129], logits[1, 0], logits[2, 64] = 9.0, 9.0, 9.0
    w1 = torch.zeros((E, K, 2 * F), dtype=BF16, device=DEV)
    w2 = torch.zeros((E, F, 64), dtype=BF16, device=DEV)
    for e in (0, 64, 129):
        w1[e], w2[e] = randn(gen(e), K, 2 * F, scale=K ** -0.5).to(DEV), randn(gen(e + 1), F, 64, scale=F ** -0.5).to(DEV)
    got = gc.moe_layer(x.to(DEV), logits.to(DEV), w1, w2, 1)
    for t, e in ((0, 129), (1, 0), (2, 64)):
        one = torch.zeros((1, 1))
        ref.check(got[t:t + 1], *ref.layer(x[t:t + 1], one, w1[e:e + 1].cpu(), w2[e:e + 1].cpu(), 1), f"expert {e}")


@pytest.mark.parametrize("op", ["norm", "norm fp8", "rows", "blocks", "layer"])
def test_outputs_in_larger_buffers(op):
    """Outputs of the caller's own are written whole and nothing beside them is."""
    g = gen(21)
    M, N = 13, 272
    x, res, w = dev(randn(g, M, N), randn(g, M, N), randn(g, N))
    buf, fbuf = filled(M + 2, N), torch.full((M + 2, 8), 7.0, device=DEV)
    codes = torch.full((M + 2, N), 0x55, dtype=torch.uint8, device=DEV)
    out, q, s = buf[1:M + 1], codes[1:M + 1].view(E4M3), fbuf[1:M + 1, 2:5]
    if op == "norm":
        got = gc.rms_norm(x, w, residual=res, out=out)
        assert got.y is out and torch.equal(out, gc.rms_norm(x, w, residual=res).y)
    elif op == "norm fp8":
        got, want = gc.rms_norm(x, w, residual=res, out=q, scales=s, fp8=True), gc.rms_norm(x, w, residual=res, fp8=True)
        assert got.y is q and got.scales is s
        assert torch.equal(codes[1:M + 1], want.y.view(torch.uint8)) and torch.equal(s, want.scales)
    elif op == "rows":
        got, want = gc.quantize_fp8(x, out=q, scales=s), gc.quantize_fp8(x)
        assert got.q is q and torch.equal(codes[1:M + 1], want.q.view(torch.uint8)) and torch.equal(s, want.scales)
    elif op == "blocks":
        gc.quantize_fp8(x, block_rows=128, out=q)
        assert torch.equal(codes[1:M + 1], gc.quantize_fp8(x, block_rows=128).q.view(torch.uint8))
    else:
        ins = dev(*layer_inputs(M, 6, 2, 64, 40, N, 3)[:4])
        assert torch.equal(gc.moe_layer(*ins, 2, out=out), gc.moe_layer(*ins, 2))
    assert (buf.view(torch.int16)[[0, M + 1]] == SENTINEL).all()
    assert (codes[[0, M + 1]] == 0x55).all()
    assert (fbuf[[0, M + 1]] == 7.0).all() and (fbuf[:, :2] == 7.0).all() and (fbuf[:, 5:] == 7.0).all()


def test_refusals():
    g = gen(2)
    x, res, w = dev(randn(g, 6, 64), randn(g, 6, 64), randn(g, 64))
    q, s = gc.quantize_fp8(x)
    b, bs = gc.quantize_fp8(x, block_rows=128)
    wide = dev(randn(g, 6, 128))[0]
    for call, what in ((lambda: gc.rms_norm(wide[:, ::2], w), "contiguous"), (lambda: gc.rms_norm(x, w[:32]), "weight"),
                       (lambda: gc.rms_norm(x, w, residual=res[:5]), "residual"),
                       (lambda: gc.rms_norm(x, w, partials=res), "partials"),
                       (lambda: gc.rms_norm(x, w, sum_out=x), "sum_out"), (lambda: gc.rms_norm(x, w, scales=s), "fp8"),
                       (lambda: gc.rms_norm(x, w, fp8=True, scales=s.expand(6, 1)[:5]), "scales"),
                       (lambda: gc.rms_norm(x, w, fp8=True, scales=torch.zeros(1, device=DEV).expand(6, 1)), "apart"),
                       (lambda: gc.quantize_fp8(x, block_rows=64), "block_rows"),
                       (lambda: gc.gemm_fp8(q, s[:5], b, bs), "a_scales"), (lambda: gc.gemm_fp8(q, s, b, s), "b_scales"),
                       (lambda: gc.gemm_fp8(q, s.cpu(), b, bs), "device"), (lambda: gc.gemm_fp8(q, s, b[:, :48], bs), "B"),
                       (lambda: gc.gemm_fp8(q, s, b, bs, out=x), "out"),
                       (lambda: gc.moe_layer(x, s, x[None], x[None], 1), "w1"),
                       (lambda: gc.moe_layer(x, s[:5], x[None], x[None], 1), "logits")):
        with pytest.raises(ValueError, match=what):
            call()
    for call in (lambda: gc.rms_norm(x, w.half()), lambda: gc.rms_norm(x, w, out=q), lambda: gc.quantize_fp8(q),
                 lambda: gc.gemm_fp8(x, s, b, bs), lambda: gc.rms_norm(x, w, residual=res.float())):
        with pytest.raises(TypeError):
            call()
    ins = dev(*layer_inputs(4, 6, 2, 64, 40, 64, 3)[:4])
    many = dev(*layer_inputs(17, 6, 2, 64, 40, 64, 3)[:4])
    small = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    for call in (lambda: gc.rms_norm(x, w, eps=-1.0), lambda: gc.rms_norm(x, w, residual=res, out=x, sum_out=x),
                 lambda: gc.moe_layer(*ins, 2, workspace=False), lambda: gc.moe_layer(*ins, 2, workspace=small),
                 lambda: gc.moe_layer(*ins, 2, first=1), lambda: gc.moe_layer(*many, 2), lambda: gc.moe_layer(*ins, 17),
                 lambda: gc.gemm_fp8(q, s, b[:4].contiguous(), bs), lambda: gc.quantize_fp8(x[:, :8].contiguous()),
                 lambda: gc.gemm_fp8(q, s, torch.cat([b, b[:2]]), bs, workspace=small), lambda: gc.moe_layer(*ins, 0)):
        with pytest.raises(RuntimeError):
            call()


def test_workspaces_of_the_callers_own():
    ops = operands(500, 4104, 4112, 4)
    ws = torch.zeros(gc.grouped_workspace_bytes(), dtype=torch.uint8, device=DEV)
    assert torch.equal(gc.gemm_fp8(*ops, workspace=ws), gc.gemm_fp8(*ops))
    ins = dev(*layer_inputs(5, 12, 3, 264, 72, 136, 3)[:4])
    assert torch.equal(gc.moe_layer(*ins, 3, workspace=ws), gc.moe_layer(*ins, 3))
    # (the counters are left at zero: a grouped product may take it next)
    w = ins[2]
    off = torch.tensor([0] * 5 + [5] * 8, dtype=torch.int32, device=DEV)
    assert torch.equal(gc.grouped_gemm(ins[0], w, off, workspace=ws), gc.grouped_gemm(ins[0], w, off))
    assert (ws[:4096] == 0).all()
