"""Host-side checks of include/gemm_coll_grouped.h (no GPU needed): every
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
HEADER = os.path.join(ROOT, "include", "gemm_coll_grouped.h")
P = 0x7F0000000000         # well-formed addresses that nothing reads


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gc.LIB_PATH):
        from tensor_bf16_gemm_amd import build
        build.build()
    return gc.lib()


def test_exports_every_declared_function(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int(?:64_t)?\s+(gemm_coll_\w+)\s*\(", text, flags=re.M))
    assert names == {"gemm_coll_grouped_workspace_bytes", "gemm_coll_moe_route", "gemm_coll_group_rows",
                     "gemm_coll_grouped_gemm", "gemm_coll_moe_combine", "gemm_coll_lora_add",
                     "gemm_coll_lora_workspace_bytes", "gemm_coll_grouped_plan"}
    out = subprocess.run(["nm", "-D", "--defined-only", gc.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= {l.split()[-1] for l in out.splitlines() if " T " in l}


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemm_coll_grouped.h"\nint main(void){return 0;}\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


def route(L, **kw):
    a = dict(logits=P, type=0, stride=64, T=300, E=64, k=8, score=0, bias=None, renorm=1, scale=1.0,
             ids=P, weights=P, offsets=P, rows=P, slots=P, ws=P, wb=1 << 30)
    a.update(kw)
    return L.gemm_coll_moe_route(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(E=1025, stride=1025), dict(k=0), dict(k=17),
                                dict(stride=63), dict(type=2), dict(type=-1), dict(score=2),
                                dict(logits=None), dict(logits=P + 2), dict(ids=None), dict(ids=P + 1),
                                dict(weights=None), dict(offsets=None), dict(rows=None), dict(slots=None),
                                dict(rows=P + 2), dict(bias=P + 1), dict(ws=None), dict(ws=P + 8),
                                dict(wb=4096)])
def test_route_refuses(L, kw):
    assert route(L, **kw) == gc.GC_EINVAL


def test_route_sizes(L):
    assert route(L, T=(1 << 24) // 8 + 1) == gc.GC_ENOTSUP
    assert route(L, T=0, offsets=None, rows=None, slots=None, logits=None, ids=None, weights=None) == gc.GC_OK


@pytest.mark.parametrize("kw,code", [(dict(T=-1), gc.GC_EINVAL), (dict(k=0), gc.GC_EINVAL),
                                     (dict(groups=0), gc.GC_EINVAL), (dict(groups=1025), gc.GC_EINVAL),
                                     (dict(offsets=None), gc.GC_EINVAL), (dict(ids=None), gc.GC_EINVAL),
                                     (dict(rows=P + 1), gc.GC_EINVAL), (dict(slots=None), gc.GC_EINVAL),
                                     (dict(T=2000, ws=None), gc.GC_EINVAL),
                                     (dict(T=(1 << 24) + 1), gc.GC_ENOTSUP)])
def test_group_rows_refuses(L, kw, code):
    a = dict(ids=P, T=2000, k=1, groups=8, offsets=P, rows=P, slots=P, ws=P, wb=1 << 30)
    a.update(kw)
    assert L.gemm_coll_group_rows(*a.values(), None) == code


def gemm(L, **kw):
    a = dict(X=P, T=100, W=P, offsets=P, rows=P, S=200, K=64, N=64, E=4, act=0, out=P, ws=None, wb=0)
    a.update(kw)
    return L.gemm_coll_grouped_gemm(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(S=-1), dict(K=-8), dict(N=-8), dict(K=4), dict(N=12),
                                dict(E=0), dict(E=1025), dict(act=2), dict(act=-1), dict(N=24, act=1),
                                dict(rows=None), dict(X=None), dict(X=P + 8), dict(W=None), dict(W=P + 2),
                                dict(out=None), dict(out=P + 4), dict(offsets=None), dict(offsets=P + 2),
                                dict(rows=P + 1)])
def test_grouped_gemm_refuses(L, kw):
    assert gemm(L, **kw) == gc.GC_EINVAL


@pytest.mark.parametrize("kw", [dict(T=1 << 24), dict(S=1 << 24), dict(K=1 << 15, N=1 << 15),
                                dict(T=1 << 32), dict(K=1 << 40), dict(K=8, N=(1 << 24) + 8)])
def test_grouped_gemm_too_large(L, kw):
    assert gemm(L, **{**dict(S=100, rows=P), **kw}) == gc.GC_ENOTSUP


def test_grouped_gemm_nothing_to_do(L):
    assert gemm(L, S=0, out=None, offsets=None) == gc.GC_OK
    assert gemm(L, N=0, out=None) == gc.GC_OK


@pytest.mark.parametrize("kw,code", [(dict(S=-1), gc.GC_EINVAL), (dict(T=-1), gc.GC_EINVAL),
                                     (dict(k=0), gc.GC_EINVAL), (dict(k=17), gc.GC_EINVAL),
                                     (dict(N=12), gc.GC_EINVAL), (dict(npeers=16), gc.GC_EINVAL),
                                     (dict(npeers=-1), gc.GC_EINVAL), (dict(partials=None), gc.GC_EINVAL),
                                     (dict(partials=P + 8), gc.GC_EINVAL), (dict(stride=1004), gc.GC_EINVAL),
                                     (dict(stride=632), gc.GC_EINVAL), (dict(Y=None), gc.GC_EINVAL),
                                     (dict(slots=None), gc.GC_EINVAL), (dict(weights=P + 2), gc.GC_EINVAL),
                                     (dict(out=P + 8), gc.GC_EINVAL), (dict(T=1 << 31), gc.GC_ENOTSUP),
                                     (dict(T=0, out=None), gc.GC_OK), (dict(N=0, out=None), gc.GC_OK)])
def test_combine_refuses(L, kw, code):
    a = dict(Y=P, S=30, slots=P, weights=P, T=10, k=3, N=64, partials=P, npeers=2, stride=640, out=P)
    a.update(kw)
    assert L.gemm_coll_moe_combine(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [(dict(M=-1), gc.GC_EINVAL), (dict(K=12), gc.GC_EINVAL),
                                     (dict(N=20), gc.GC_EINVAL), (dict(r=0), gc.GC_EINVAL),
                                     (dict(r=12), gc.GC_EINVAL), (dict(r=136), gc.GC_EINVAL),
                                     (dict(G=0), gc.GC_EINVAL), (dict(G=1024), gc.GC_EINVAL),
                                     (dict(base=None), gc.GC_EINVAL), (dict(X=P + 8), gc.GC_EINVAL),
                                     (dict(down=None), gc.GC_EINVAL), (dict(up=P + 2), gc.GC_EINVAL),
                                     (dict(scale=None), gc.GC_EINVAL), (dict(offsets=P + 1), gc.GC_EINVAL),
                                     (dict(rows=None), gc.GC_EINVAL), (dict(out=None), gc.GC_EINVAL),
                                     (dict(M=1 << 24), gc.GC_ENOTSUP), (dict(M=0, out=None), gc.GC_OK)])
def test_lora_refuses(L, kw, code):
    a = dict(base=P, X=P, down=P, up=P, scale=P, offsets=P, rows=P, M=20, K=64, N=64, r=16, G=4, out=P,
             ws=P, wb=1 << 30)
    a.update(kw)
    assert L.gemm_coll_lora_add(*a.values(), None) == code


def test_binding_refuses_wrong_tensors():
    bf, i32 = torch.bfloat16, torch.int32
    X, W = torch.zeros(4, 16, dtype=bf), torch.zeros(2, 16, 32, dtype=bf)
    off = torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="device"):
        gc.grouped_gemm(X, W, off)
    with pytest.raises(TypeError, match="bfloat16"):
        gc.grouped_gemm(X.float(), W, off)
    with pytest.raises(ValueError, match="act"):
        gc.grouped_gemm(X, W, off, act="relu")
    with pytest.raises(ValueError, match="W"):
        gc.grouped_gemm(X, W[0], off)
    with pytest.raises(TypeError, match="logits"):
        gc.moe_route(torch.zeros(4, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="device"):
        gc.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="ids"):
        gc.group_rows(torch.zeros((1, 2, 3), dtype=i32), 4)
    with pytest.raises(TypeError, match="ids"):
        gc.group_rows(torch.zeros(4), 4)
    with pytest.raises(ValueError, match="slots"):
        gc.moe_combine(X, off, torch.zeros(3))
    with pytest.raises(ValueError, match="down"):
        gc.lora_add(X, X, W[0], W, torch.zeros(2), off, off)


def test_grouped_plan():
    """The way products are run changes with the sizes as measured: few rows stream, many groups
    and tall ones take tiles, few tall groups tiles split along K (never without workspace)."""
    plan = gc.grouped_plan
    assert plan(8, 7168, 1792, 64, act="silu_glu") == dict(tiles=0, splits=1, block_rows=16)
    assert plan(64, 7168, 1792, 8)["block_rows"] == 16
    assert plan(128, 7168, 1792, 8)["block_rows"] == 32
    assert plan(512, 7168, 1792, 8)["block_rows"] == 64
    assert plan(512, 7168, 1792, 64, act="silu_glu") == dict(tiles=1, splits=1, block_rows=0)
    few = plan(2048, 7168, 1792, 8)
    assert few["tiles"] == 1 and few["splits"] > 1
    assert plan(2048, 7168, 1792, 8, workspace=False)["splits"] == 1
    assert plan(32768, 7168, 1792, 64, act="silu_glu")["splits"] == 1
    assert plan(0, 64, 64, 4) == dict(tiles=0, splits=1, block_rows=0)
    for bad in (dict(S=-1), dict(K=4), dict(N=12), dict(E=0), dict(E=1025), dict(cus=0)):
        with pytest.raises(RuntimeError):
            plan(**{**dict(S=8, K=64, N=64, E=4), **bad})


def test_plan_struct_layout(tmp_path):
    from tensor_bf16_gemm_amd.grouped import GroupedPlan
    names = [n for n, _ in GroupedPlan._fields_]
    src = tmp_path / "plan.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gemm_coll_grouped.h"\nint main(void){'
                   + "".join(f'printf("%zu ", offsetof(gc_grouped_plan,{n}));' for n in names)
                   + 'printf("%zu\\n", sizeof(gc_grouped_plan)); return 0;}\n')
    exe = tmp_path / "plan"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(GroupedPlan, n).offset for n in names] + [ctypes.sizeof(GroupedPlan)]
