"""The operators between and around the projections on streams of their own, on
two streams at once, and on tensors that are not on the current device."""
import pytest
import torch

import tensor_bf16_gemm_amd as gc
from gpu_util import log
from test_devices_gpu import Elsewhere
from test_streams_gpu import BUSY, bytes_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
M, N, K, E = 192, 1024, 512, 6


def randn(*shape, dtype=BF):
    return torch.randn(shape, device=DEV, dtype=F32).to(dtype)


def flat(r):
    return [r] if isinstance(r, torch.Tensor) else [t for t in r if t is not None]


def raw(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def same(a, b):
    return len(flat(a)) == len(flat(b)) and all(torch.equal(raw(x), raw(y)) for x, y in zip(flat(a), flat(b)))


def product():
    a, sa = gc.quantize_fp8(randn(M, K))
    b, sb = gc.quantize_fp8(randn(N, K), block_rows=128)
    return a, sa, b, sb, randn(3, M, N)


def deep():
    """Cut along K, so that it uses the workspace."""
    a, sa = gc.quantize_fp8(randn(500, 4096))
    b, sb = gc.quantize_fp8(randn(4104, 4096), block_rows=128)
    return a, sa, b, sb, randn(2, 500, 4104)


# name: (inputs, call(inputs, stream))
CALLS = {
    "rms_norm": (lambda: (randn(M, N), randn(N), randn(M, N), randn(2, M, N)),
                 lambda a, s: gc.rms_norm(a[0], a[1], residual=a[2], partials=a[3], fp8=True, stream=s)),
    "rms_norm alone": (lambda: (randn(M, N), randn(N, dtype=F32)), lambda a, s: gc.rms_norm(*a, stream=s)),
    "quantize_fp8": (lambda: (randn(M, N),), lambda a, s: gc.quantize_fp8(a[0], stream=s)),
    "gemm_fp8": (product, lambda a, s: gc.gemm_fp8(*a, stream=s)),
    "gemm_fp8 cut": (deep, lambda a, s: gc.gemm_fp8(*a, stream=s)),
    "moe_layer": (lambda: (randn(9, K), randn(9, E, dtype=F32), randn(E, K, 256), randn(E, 128, N), randn(2, 9, N)),
                  lambda a, s: gc.moe_layer(*a[:4], 2, partials=a[4], stream=s)),
}


@pytest.fixture(scope="module")
def side():
    return torch.cuda.Stream()


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_come_from_the_stream_of_the_call(name, side):
    make, call = CALLS[name]
    a = make()
    with torch.cuda.stream(side):
        want = [t.clone() for t in flat(call(a, None))]
    torch.cuda.synchronize()
    sizes = {bytes_of(t) for t in flat(call(a, None))}
    torch.cuda.synchronize()
    log(f"{name}: outputs of {sorted(sizes)} bytes")
    freed = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    at = {t.untyped_storage().data_ptr() for t in freed}
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in freed]
    del freed
    got = flat(call(a, side))
    assert not at & {t.untyped_storage().data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.all(c == 7) for c in copies)
    assert same(got, want)


@pytest.mark.parametrize("name", list(CALLS))
def test_inputs_outlive_a_call_on_another_stream(name, side):
    make, call = CALLS[name]
    torch.manual_seed(5)
    a = make()
    with torch.cuda.stream(side):
        want = [t.clone() for t in flat(call([t.clone() for t in a], None))]
    torch.cuda.synchronize()
    log(name)
    big = [t for t in a if bytes_of(t) > 4096]
    at, sizes = {t.data_ptr() for t in big}, [bytes_of(t) for t in big]
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = flat(call(a, side))
    del a, big
    again = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    assert not at & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", list(CALLS))
def test_raw_handle_and_current_stream(name, side):
    make, call = CALLS[name]
    a = make()
    want = [t.clone() for t in flat(call(a, None))]
    torch.cuda.synchronize()
    for s in (side.cuda_stream, torch.cuda.current_stream(), side):
        got = flat(call(a, s))
        torch.cuda.synchronize()
        assert same(got, want)
    with torch.cuda.stream(side):
        got = flat(call(a, 0))
        torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", ["gemm_fp8 cut", "moe_layer"])
def test_two_streams_at_once(name, side):
    """Calls in flight on two streams have workspaces of their own."""
    make, call = CALLS[name]
    a, b = make(), make()
    want = [[t.clone() for t in flat(call(x, None))] for x in (a, b)]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20000)
        with torch.cuda.stream(other):
            torch.cuda._sleep(20000)
        got = [call(a, side), call(b, other)]
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


@pytest.mark.parametrize("name", list(CALLS))
def test_captured(name, side):
    """A graph of one call, replayed with new inputs and the program's own calls between."""
    make, call = CALLS[name]
    a = make()
    with torch.cuda.stream(side):
        call(a, None)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call(a, None)
        for _ in range(3):
            for t, n in zip(a, make()):
                t.copy_(n)
            graph.replay()
            torch.cuda.synchronize()
            assert same(out, call(a, None))
            torch.cuda.synchronize()


ARGS = [
    (lambda x, w, r, y, s, m: gc.rms_norm(x, w, residual=r, out=y, scales=s, sum_out=m, fp8=True),
     [("x", (4, 64), BF), ("weight", (64,), BF), ("residual", (4, 64), BF), ("out", (4, 64), E4M3),
      ("scales", (4, 1), F32), ("sum_out", (4, 64), BF)]),
    (lambda x, q, s: gc.quantize_fp8(x, out=q, scales=s),
     [("x", (4, 64), BF), ("out", (4, 64), E4M3), ("scales", (4, 1), F32)]),
    (gc.gemm_fp8, [("A", (4, 64), E4M3), ("a_scales", (4, 1), F32), ("B", (8, 64), E4M3), ("b_scales", (1, 1), F32),
                   None, ("out", (4, 8), BF)]),
    (lambda x, l, a, b, c, o: gc.moe_layer(x, l, a, b, 2, bias=c, out=o),
     [("x", (4, 16), BF), ("logits", (4, 3), F32), ("w1", (3, 16, 32), BF), ("w2", (3, 16, 8), BF),
      ("bias", (3,), F32), ("out", (4, 8), BF)])]


@pytest.mark.parametrize("call,args,which", [(c, a, x[0]) for c, a in ARGS for x in a if x])
def test_tensors_of_another_device_are_refused(call, args, which):
    def make(x):
        if not x:
            return x
        return Elsewhere(x[1], x[2]) if x[0] == which else torch.zeros(x[1], dtype=x[2], device="cuda")
    with pytest.raises(ValueError, match=f"{which} is on cuda:1"):
        call(*[make(x) for x in args])
