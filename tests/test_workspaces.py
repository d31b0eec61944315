"""Default workspaces made by several threads at once, and workspaces of the
caller's own (no GPU needed: the device calls are stood in for)."""
import threading
import time

import pytest
import torch

import tensor_bf16_gemm_amd as gc
from tensor_bf16_gemm_amd import grouped

THREADS = 8


def at_once(f):
    """Results of f() in several threads that start together."""
    start, got = threading.Barrier(THREADS), [None] * THREADS

    def work(i):
        start.wait()
        got[i] = f()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return got


@pytest.fixture
def no_device(monkeypatch):
    """grouped's workspaces on host memory; the synchronization only lets other threads run."""
    made = []
    zeros = torch.zeros

    def host_zeros(n, dtype, device):
        made.append(zeros(n, dtype=dtype))
        return made[-1]
    monkeypatch.setattr(grouped, "_scratch", {})
    monkeypatch.setattr(grouped, "_kept", [])
    monkeypatch.setattr(grouped, "_base_bytes", {0: 4096})
    monkeypatch.setattr(torch, "zeros", host_zeros)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d=None: time.sleep(0.05))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    return made


def kept(pointer):
    """Whether the memory at `pointer` is held by the module."""
    return pointer in {t.data_ptr() for t in grouped._kept} | {t[1] for t in grouped._scratch.values()}


def test_threads_share_the_first_workspace_of_a_stream(no_device):
    got = at_once(lambda: grouped._workspace(None, 7))
    assert len(no_device) == 1
    assert set(got) == {(no_device[0].data_ptr(), 4096)}


def test_threads_that_grow_a_workspace(no_device):
    """Every pointer handed out stays allocated, with the bytes it was handed out for."""
    grouped._workspace(None, 7)
    got = at_once(lambda: grouped._workspace(None, 7, 1000))
    assert all(n >= 4096 + 1000 and kept(p) for p, n in got)
    assert len(no_device) == 2 and len(set(got)) == 1
    a = grouped._workspace(None, 7, 1001)
    assert a[1] >= 4096 + 2000 and kept(a[0]) and kept(got[0][0])
    assert grouped._workspace(None, 7, 500) == a
    assert grouped._workspace(None, 8)[0] != a[0]


def test_threads_share_the_projections_workspace(monkeypatch):
    monkeypatch.setattr(gc, "_workspaces", {})
    made = []

    def make():
        time.sleep(0.05)
        made.append(object())
        return made[-1]
    got = at_once(lambda: gc._cached_workspace((0, 7), make))
    assert len(made) == 1 and all(w is made[0] for w in got)


def test_workspaces_in_host_memory_are_refused():
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        grouped._workspace(ws, 0)
    with pytest.raises(ValueError, match="device tensor"):
        gc._ws_fields(ws, None, 0)
