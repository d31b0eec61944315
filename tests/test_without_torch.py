"""What the package does without tensors needs the library alone: neither
torch nor the extension module (no GPU needed)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, **env), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-800:]
    return r.stdout


@pytest.mark.parametrize("call", ["plan('ar', 4096, 6288, 7168, 8)", "should_run(128)", "strerror(-22)"])
@pytest.mark.parametrize("missing", ["torch", "tensor_bf16_gemm_amd._native"])
def test_library_alone(call, missing):
    code = f"import sys; sys.modules[{missing!r}] = None; import tensor_bf16_gemm_amd as gc; print(gc.{call})"
    assert run(code) == run(f"import tensor_bf16_gemm_amd as gc; print(gc.{call})")


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_build_puts_the_library_in_place_first(missing, tmp_path):
    """Without PyTorch or a host compiler the binding's failure is reported after the library is there.
    (The compilers are stood in for: hipcc by one that touches its output.)"""
    hipcc = tmp_path / "hipcc"
    hipcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho built > "$2"\n')
    hipcc.chmod(0o755)
    code = f"""
import sys
if {missing!r} == "torch":
    sys.modules["torch"] = None
from tensor_bf16_gemm_amd import build as b
b.LIB, b.NATIVE, b.PKG = {str(tmp_path)!r} + "/libgemm_coll.so", {str(tmp_path)!r} + "/_native.so", {str(tmp_path)!r}
try:
    b.build(b.LIB)
except RuntimeError as e:
    print("refused", "binding" in str(e), open(b.LIB).read().strip())
"""
    path = os.environ["PATH"]
    if missing == "g++":
        (tmp_path / "bin").mkdir()
        path = str(tmp_path / "bin")
    assert run(code, PATH=path, HIPCC=str(hipcc)).split() == ["refused", "True", "built"]
