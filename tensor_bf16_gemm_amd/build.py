"""Build the HIP library ``libgemm_coll.so`` for gfx950 and the binding
``_native.so``, in-tree.

    python -m tensor_bf16_gemm_amd.build

Compiles csrc/gemm_coll.hip and csrc/grouped.hip (host C ABI + device
kernels), each in a hipcc of its own, and links them into
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
SOURCES = ("gemm_coll.hip", "grouped.hip")


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


def _run(cmds: list[list[str]]):
    """Runs the commands side by side; raises with the output of the first that failed."""
    runs = [(c, subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
            for c in cmds]
    for cmd, p in [(c, (p, p.communicate()[0])) for c, p in runs]:
        if p[0].returncode != 0:
            raise RuntimeError(f"build failed:\n{' '.join(cmd)}\n{p[1]}")


def build(out_path: str = LIB, extra: tuple[str, ...] = ()) -> str:
    """Compile the library and, at its own place, the binding (always); returns the library's path."""
    with tempfile.TemporaryDirectory(dir=os.path.dirname(out_path)) as tmp:
        objs = [os.path.join(tmp, name + ".o") for name in SOURCES]
        cmds = [[hipcc(), *compile_flags(), "-c", *extra, "-o", o, os.path.join(CSRC, name)]
                for o, name in zip(objs, SOURCES)]
        binding = out_path == LIB
        if binding:
            flags, libs = binding_flags()
            cmds.append(["g++", *flags, "-c", "-o", os.path.join(tmp, "binding.o"),
                         os.path.join(CSRC, "binding.cpp")])
        _run(cmds)
        lib = os.path.join(tmp, "libgemm_coll.so")
        _run([[hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", lib, *objs]])
        if binding:
            native = os.path.join(tmp, "_native.so")
            _run([["g++", "-shared", "-o", native, os.path.join(tmp, "binding.o"), f"-L{tmp}",
                   "-l:libgemm_coll.so", *libs]])
            os.replace(native, NATIVE)
        os.replace(lib, out_path)
    return out_path


if __name__ == "__main__":
    print(build())
