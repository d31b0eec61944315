"""Build the HIP library ``libgemm_coll.so`` for gfx950 and the binding
``_native.so``, in-tree.

    python -m tensor_bf16_gemm_amd.build

Compiles csrc/gemm_coll.hip, csrc/grouped.hip and csrc/layer.hip (host C ABI +
device kernels), each in a hipcc of its own, and links them into
``tensor_bf16_gemm_amd/libgemm_coll.so``; csrc/binding.cpp (the tensor side of
the routed and grouped operators, host code against PyTorch's headers) becomes
``tensor_bf16_gemm_amd/_native.so``, which finds the library beside itself.
Packed-fp32 VALU instructions are disabled for device code
(-packed-fp32-ops); hipcc's host pass warns that it does not know that
feature, which is harmless.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgemm_coll.so")
NATIVE = os.path.join(PKG, "_native.so")
ARCH = "gfx950"
SOURCES = ("gemm_coll.hip", "grouped.hip", "layer.hip")


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build the library)")


def compile_flags() -> list[str]:
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            f"-I{INCLUDE}", f"-I{CSRC}"]


def binding_flags() -> tuple[list[str], list[str]]:
    """Compiler and linker flags of the binding (PyTorch's headers and libraries)."""
    import torch
    at = os.path.dirname(torch.__file__)
    return (["-O2", "-std=c++17", "-fPIC", "-Wall",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
             f"-I{at}/include", f"-I{at}/include/torch/csrc/api/include",
             f"-I{sysconfig.get_paths()['include']}"],
            [f"-L{at}/lib", "-lc10", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])


def _start(cmd: list[str]):
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _wait(runs):
    """Waits for the commands that run side by side; raises with the output of the first that failed."""
    for cmd, p, text in [(c, p, p.communicate()[0]) for c, p in runs]:
        if p.returncode != 0:
            raise RuntimeError(f"build failed:\n{' '.join(cmd)}\n{text}")


def _compile_binding(tmp: str):
    """The running compilation of the binding, or why there is none (no g++, no PyTorch)."""
    try:
        return _start(["g++", *binding_flags()[0], "-c", "-o", os.path.join(tmp, "binding.o"),
                       os.path.join(CSRC, "binding.cpp")])
    except (ImportError, OSError) as e:
        return e


def _link_binding(run, tmp: str):
    if isinstance(run, Exception):
        raise RuntimeError(f"{LIB} is built, its binding {NATIVE} is not: {run}") from run
    _wait([run])
    native = os.path.join(tmp, "_native.so")
    _wait([_start(["g++", "-shared", "-o", native, os.path.join(tmp, "binding.o"), f"-L{PKG}",
                   "-l:libgemm_coll.so", *binding_flags()[1]])])
    os.replace(native, NATIVE)


def build(out_path: str = LIB, extra: tuple[str, ...] = ()) -> str:
    """Compile the library and, at its own place, the binding (always); returns the library's path.
    The library is in place before the binding is asked for: it needs neither g++ nor PyTorch, and
    neither does what the package does without tensors."""
    with tempfile.TemporaryDirectory(dir=os.path.dirname(out_path)) as tmp:
        binding = _compile_binding(tmp) if out_path == LIB else None
        try:
            objs = [os.path.join(tmp, name + ".o") for name in SOURCES]
            _wait([_start([hipcc(), *compile_flags(), "-c", *extra, "-o", o, os.path.join(CSRC, name)])
                   for o, name in zip(objs, SOURCES)])
            lib = os.path.join(tmp, "libgemm_coll.so")
            _wait([_start([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", lib, *objs])])
            os.replace(lib, out_path)
        except BaseException:
            if isinstance(binding, tuple):
                binding[1].kill()
                binding[1].communicate()
            raise
        if binding is not None:
            _link_binding(binding, tmp)
    return out_path


if __name__ == "__main__":
    print(build())
