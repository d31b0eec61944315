"""Host-side checks of include/gemm_coll_layer.h (no GPU needed): every
declared function is exported, and invalid arguments are refused before any
HIP call; the binding refuses wrong tensors."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import tensor_bf16_gemm_amd as gc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_coll_layer.h")
P = 0x7F0000000000         # well-formed addresses that nothing reads
EINVAL, ENOTSUP, OK = gc.GC_EINVAL, gc.GC_ENOTSUP, gc.GC_OK
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gc.LIB_PATH):
        from tensor_bf16_gemm_amd import build
        build.build()
    return gc.lib()


def test_exports_every_declared_function(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int(?:64_t)?\s+(gemm_coll_\w+)\s*\(", text, flags=re.M))
    assert names == {"gemm_coll_rms_norm", "gemm_coll_quantize_fp8", "gemm_coll_gemm_fp8",
                     "gemm_coll_gemm_fp8_plan", "gemm_coll_moe_layer"}
    out = subprocess.run(["nm", "-D", "--defined-only", gc.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= {l.split()[-1] for l in out.splitlines() if " T " in l}


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemm_coll_layer.h"\nint main(void){return 0;}\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


@pytest.mark.parametrize("kw,code", [(dict(M=-1), EINVAL), (dict(N=-8), EINVAL), (dict(N=20), EINVAL),
                                     (dict(N=72), EINVAL), (dict(npeers=-1), EINVAL), (dict(npeers=16), EINVAL),
                                     (dict(partials=None), EINVAL), (dict(partials=P + 8), EINVAL),
                                     (dict(stride=636), EINVAL), (dict(stride=632), EINVAL), (dict(x=None), EINVAL),
                                     (dict(x=P + 8), EINVAL), (dict(residual=P + 2), EINVAL),
                                     (dict(weight=None), EINVAL), (dict(weight=P + 4), EINVAL), (dict(type=2), EINVAL),
                                     (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL), (dict(sum=P + 8), EINVAL),
                                     (dict(codes=P + 8), EINVAL), (dict(scales=None), EINVAL),
                                     (dict(scales=P + 2), EINVAL), (dict(ss=0), EINVAL),
                                     (dict(codes=None, y=None), EINVAL), (dict(codes=None, y=P + 2), EINVAL),
                                     (dict(codes=None, y=P + 64, sum=P + 64), EINVAL),
                                     (dict(M=1 << 30), ENOTSUP), (dict(N=1 << 16, ss=512), ENOTSUP),
                                     (dict(M=0, x=None), OK), (dict(N=0, x=None), OK)])
def test_rms_norm_refuses(L, kw, code):
    a = dict(x=P, residual=P, partials=P, npeers=2, stride=640, weight=P, type=1, eps=1e-6, M=10, N=64, sum=P, y=None,
             codes=P, scales=P, ss=1)
    a.update(kw)
    assert L.gemm_coll_rms_norm(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [(dict(M=-1), EINVAL), (dict(K=-16), EINVAL), (dict(K=24), EINVAL),
                                     (dict(rows=0), EINVAL), (dict(rows=64), EINVAL), (dict(x=None), EINVAL),
                                     (dict(x=P + 8), EINVAL), (dict(codes=None), EINVAL), (dict(codes=P + 8), EINVAL),
                                     (dict(scales=None), EINVAL), (dict(scales=P + 1), EINVAL), (dict(ss=1), EINVAL),
                                     (dict(M=1 << 31), ENOTSUP), (dict(K=1 << 31, ss=1 << 30), ENOTSUP),
                                     (dict(M=0, x=None), OK), (dict(K=0, x=None), OK)])
def test_quantize_refuses(L, kw, code):
    a = dict(x=P, M=10, K=144, rows=1, codes=P, scales=P, ss=2)
    a.update(kw)
    assert L.gemm_coll_quantize_fp8(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [(dict(M=-1), EINVAL), (dict(N=-8), EINVAL), (dict(N=12), EINVAL),
                                     (dict(K=8), EINVAL), (dict(K=-16), EINVAL), (dict(A=None), EINVAL),
                                     (dict(A=P + 8), EINVAL), (dict(sa=None), EINVAL), (dict(sa=P + 2), EINVAL),
                                     (dict(row=-1), EINVAL), (dict(block=-1), EINVAL), (dict(B=None), EINVAL),
                                     (dict(B=P + 1), EINVAL), (dict(sb=None), EINVAL), (dict(npeers=16), EINVAL),
                                     (dict(npeers=-1), EINVAL), (dict(partials=None), EINVAL),
                                     (dict(partials=P + 4), EINVAL), (dict(stride=7), EINVAL),
                                     (dict(stride=19992), EINVAL), (dict(out=None), EINVAL), (dict(out=P + 8), EINVAL),
                                     (dict(ws=P + 8, wb=1 << 40), EINVAL), (dict(M=1 << 24), ENOTSUP),
                                     (dict(N=1 << 24), ENOTSUP), (dict(K=1 << 30, M=2), ENOTSUP),
                                     (dict(M=1 << 20, N=1 << 11, K=16), ENOTSUP), (dict(row=1 << 29), ENOTSUP),
                                     (dict(row=1 << 23), ENOTSUP), (dict(block=1 << 40), ENOTSUP),
                                     (dict(M=0, out=None), OK), (dict(N=0, out=None), OK)])
def test_gemm_refuses(L, kw, code):
    a = dict(A=P, sa=P, row=2, block=1, B=P, sb=P, M=100, N=200, K=256, partials=P, npeers=2, stride=20000, out=P,
             ws=None, wb=0)
    a.update(kw)
    assert L.gemm_coll_gemm_fp8(*a.values(), None) == code


LAYER = dict(X=P, logits=P, type=0, stride=64, T=4, E=64, k=8, score=0, bias=None, renorm=1, scale=1.0, W1=P, W2=P,
             first=0, local=64, K=64, F=32, N=64, partials=P, npeers=2, pstride=256, out=P, ws=P, wb=1 << 40)


@pytest.mark.parametrize("kw,code", [(dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(E=1025, stride=1025), EINVAL),
                                     (dict(k=0), EINVAL), (dict(k=17), EINVAL), (dict(stride=63), EINVAL),
                                     (dict(type=2), EINVAL), (dict(score=-1), EINVAL), (dict(first=-1), EINVAL),
                                     (dict(first=1), EINVAL), (dict(local=0), EINVAL), (dict(local=65), EINVAL),
                                     (dict(first=2**31 - 1, local=2**31 - 1), EINVAL),
                                     (dict(K=12), EINVAL), (dict(F=12), EINVAL), (dict(N=12), EINVAL),
                                     (dict(K=-8), EINVAL), (dict(logits=None), EINVAL), (dict(logits=P + 2), EINVAL),
                                     (dict(bias=P + 2), EINVAL), (dict(X=None), EINVAL), (dict(X=P + 8), EINVAL),
                                     (dict(W1=None), EINVAL), (dict(W2=P + 8), EINVAL), (dict(out=P + 8), EINVAL),
                                     (dict(npeers=16), EINVAL), (dict(partials=None), EINVAL),
                                     (dict(pstride=255), EINVAL), (dict(pstride=248), EINVAL),
                                     (dict(T=17), ENOTSUP), (dict(K=1 << 26), ENOTSUP), (dict(F=1 << 24), ENOTSUP),
                                     (dict(T=16, k=16, F=(1 << 16) + 8, K=8, N=8), ENOTSUP),
                                     (dict(N=1 << 25, F=8), ENOTSUP), (dict(T=0, out=None), OK),
                                     (dict(N=0, out=None), OK)])
def test_layer_refuses(L, kw, code):
    assert L.gemm_coll_moe_layer(*{**LAYER, **kw}.values(), None) == code


def test_fp8_plan():
    """Few rows stream; many take tiles, cut along K where the tiles are few (never without workspace)."""
    plan = gc.gemm_fp8_plan
    assert plan(1, 7168, 896)["tile_cols"] < 256 and plan(16, 6288, 7168)["tile_rows"] == 16
    big = plan(4096, 6288, 7168)
    assert big["tile_cols"] == 256 and big["tile_rows"] >= 192 and big["splits"] == 1
    assert plan(256, 6288, 7168, 7)["splits"] > 1
    assert plan(256, 6288, 7168, 7, workspace=False)["splits"] == 1
    assert plan(0, 64, 64) == dict(tile_rows=0, tile_cols=0, splits=1)
    for bad in (dict(M=-1), dict(K=8), dict(N=4), dict(cus=0), dict(npeers=16)):
        with pytest.raises(RuntimeError):
            plan(**{**dict(M=8, N=64, K=64), **bad})


def test_fp8_columns_past_a_launch(L):
    """Without weights (K 0) only the columns bound a launch: refused, not planned."""
    with pytest.raises(RuntimeError):
        gc.gemm_fp8_plan(1, 1 << 28, 0)
    assert gc.gemm_fp8_plan(1, (1 << 27) - 8, 0)["tile_rows"] == 16
    assert gc.gemm_fp8_plan(1, (1 << 27) - 16, 16)["tile_rows"] == 16
    assert L.gemm_coll_gemm_fp8(None, None, 0, 0, None, None, 1, 1 << 28, 0, None, 0, 0, P, None, 0, None) == ENOTSUP


def test_plan_struct_layout(tmp_path):
    from tensor_bf16_gemm_amd.layer_abi import Fp8Plan
    names = [n for n, _ in Fp8Plan._fields_]
    src = tmp_path / "plan.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gemm_coll_layer.h"\nint main(void){'
                   + "".join(f'printf("%zu ", offsetof(gc_fp8_plan,{n}));' for n in names)
                   + 'printf("%zu\\n", sizeof(gc_fp8_plan)); return 0;}\n')
    exe = tmp_path / "plan"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(Fp8Plan, n).offset for n in names] + [ctypes.sizeof(Fp8Plan)]


def test_binding_refuses_wrong_tensors():
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    x, w = torch.zeros(4, 32, dtype=bf), torch.zeros(32)
    q, s = torch.zeros((4, 32), dtype=e4), torch.zeros((4, 1))
    with pytest.raises(ValueError, match="device"):
        gc.rms_norm(x, w)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        gc.rms_norm(x.float(), w)
    with pytest.raises(ValueError, match="x must be"):
        gc.rms_norm(x[0], w)
    with pytest.raises(ValueError, match="device"):
        gc.quantize_fp8(x)
    with pytest.raises(TypeError, match="x must be a tensor"):
        gc.layer._native.quantize_fp8(None, 1, None, None, 0)
    with pytest.raises(ValueError, match="device"):
        gc.gemm_fp8(q, s, q, s)
    with pytest.raises(TypeError, match="A must be torch.float8_e4m3fn"):
        gc.gemm_fp8(x, s, q, s)
    with pytest.raises(ValueError, match="B must be"):
        gc.gemm_fp8(q, s, q[0], s)
    with pytest.raises(ValueError, match="w1 must be"):
        gc.moe_layer(x, s, x, x, 1)
    with pytest.raises(ValueError, match="score"):
        gc.moe_layer(x, s, x[None], x[None], 1, score="relu")
    with pytest.raises(ValueError, match="device"):
        gc.moe_layer(x, s, x[None], x[None], 1)
