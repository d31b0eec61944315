"""Calls given a stream of their own: whose memory their outputs take, and how
long that of their inputs is kept.

The memory is looked at by address: the allocator hands a freed block of a
stream to the next request of that size on the same stream, whether or not
another stream still works on it."""
import pytest
import torch

import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
M, K, N, E, R = 192, 256, 1024, 4, 4
BUSY = 20_000_000          # clock ticks of a stream that is kept busy (10 ms)


def randn(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, device=DEV, dtype=torch.float32).to(dtype)


def offsets():
    return torch.tensor([0, 50, 90, 90, M], dtype=torch.int32, device=DEV)


def everybody():
    return torch.arange(M, dtype=torch.int32, device=DEV)


# name: (inputs, call(inputs, stream))
CALLS = {
    "moe_route": (lambda: (randn(M, 64, dtype=torch.float32),),
                  lambda a, s: gc.moe_route(a[0], 4, stream=s)),
    "group_rows": (lambda: (torch.randint(0, E, (M, 1), dtype=torch.int32, device=DEV),),
                   lambda a, s: gc.group_rows(a[0], E, stream=s)),
    "grouped_gemm": (lambda: (randn(M, K), randn(E, K, N), offsets()),
                     lambda a, s: gc.grouped_gemm(*a, stream=s)),
    "moe_combine": (lambda: (randn(M, N), everybody()[:, None].contiguous(), torch.ones(M, 1, device=DEV)),
                    lambda a, s: gc.moe_combine(*a, stream=s)),
    "lora_add": (lambda: (randn(M, N), randn(M, K), randn(E, K, 16), randn(E, 16, N),
                          torch.ones(E, device=DEV), offsets(), everybody()),
                 lambda a, s: gc.lora_add(*a, stream=s)),
    "gemm_ar": (lambda: (randn(M, K), randn(K, N), randn(R - 1, M, N)),
                lambda a, s: gc.gemm_ar(*a, R=R, rank=0, stream=s)),
    "gemm_rs": (lambda: (randn(M, K), randn(K, N), randn(R - 1, M, N), randn(M, N)),
                lambda a, s: gc.gemm_rs(*a, R=R, rank=1, stream=s)),
    "gemm_ar_two_shot": (lambda: (randn(M, K), randn(K, N), randn(R - 1, M, N), randn(M, N), randn(R - 1, M, N)),
                         lambda a, s: gc.gemm_ar_two_shot(*a, torch.zeros(M, N, dtype=torch.bfloat16, device=DEV),
                                                          R=R, rank=1, stream=s)),
    "peer_sum": (lambda: (randn(M, N), randn(R - 1, M, N)),
                 lambda a, s: gc.peer_sum(*a, stream=s)),
}


def flat(r):
    return [r] if isinstance(r, torch.Tensor) else list(r)


def bytes_of(t):
    return t.untyped_storage().nbytes()


@pytest.fixture(scope="module")
def side():
    return torch.cuda.Stream()


@pytest.mark.parametrize("name", [n for n in CALLS if n != "gemm_ar_two_shot"])
def test_outputs_come_from_the_stream_of_the_call(name, side):
    """A block that the current stream has freed, and that work queued there still reads, is not
    the output of a call on another stream."""
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
    torch.cuda._sleep(BUSY)                             # the current stream is busy,
    copies = [t.clone() for t in freed]                 # reads the blocks after that,
    del freed                                           # and they are free for its next request
    got = flat(call(a, side))
    assert not at & {t.untyped_storage().data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.all(c == 7) for c in copies)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("name", list(CALLS))
def test_inputs_outlive_a_call_on_another_stream(name, side):
    """Inputs dropped right after the call keep their memory until the call's stream has read them."""
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
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_outputs_outlive_their_reader_on_the_current_stream(side):
    """An output dropped after the current stream has queued its reading is not handed to the
    call's stream before."""
    make, call = CALLS["moe_combine"]
    a = make()
    out = call(a, side)
    torch.cuda.current_stream().wait_stream(side)
    at, n = out.data_ptr(), bytes_of(out)
    torch.cuda._sleep(BUSY)
    copy = out.clone()
    del out
    with torch.cuda.stream(side):
        again = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
    assert at not in {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert torch.equal(copy, call(a, None))


@pytest.mark.parametrize("name", list(CALLS))
def test_raw_handle_and_current_stream(name, side):
    """The same results through a raw handle, the default stream's, and the current stream named."""
    make, call = CALLS[name]
    a = make()
    copy = lambda: [t.clone() for t in a]  # noqa: E731
    want = flat(call(copy(), None))
    torch.cuda.synchronize()
    for s in (side.cuda_stream, torch.cuda.current_stream(), side):
        b = copy()
        torch.cuda.synchronize()
        got = flat(call(b, s))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    with torch.cuda.stream(side):
        b = copy()
        torch.cuda.synchronize()
        got = flat(call(b, 0))
        torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
