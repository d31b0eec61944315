"""ctypes side of include/gemm_coll_grouped.h: structures and signatures.  It
needs neither torch nor the extension module, as little as the library itself."""
from __future__ import annotations

import ctypes


class GroupedPlan(ctypes.Structure):
    """Mirror of ``gc_grouped_plan`` in include/gemm_coll_grouped.h."""
    _fields_ = [("tiles", ctypes.c_int32), ("splits", ctypes.c_int32), ("block_rows", ctypes.c_int32)]


def declare(L: ctypes.CDLL) -> None:
    """Sets the signatures of the functions of include/gemm_coll_grouped.h."""
    i, i64, vp, u64 = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint64
    for name, args, res in (
            ("gemm_coll_grouped_workspace_bytes", [], i64),
            ("gemm_coll_lora_workspace_bytes", [i64, i], i64),
            ("gemm_coll_moe_route", [vp, i, i64, i64, i, i, i, vp, i, ctypes.c_float, vp, vp, vp, vp,
                                     vp, vp, u64, vp], i),
            ("gemm_coll_group_rows", [vp, i64, i, i, vp, vp, vp, vp, u64, vp], i),
            ("gemm_coll_grouped_gemm", [vp, i64, vp, vp, vp, i64, i64, i64, i, i, vp, vp, u64, vp], i),
            ("gemm_coll_grouped_plan", [i64, i64, i64, i, i, i, i, ctypes.POINTER(GroupedPlan)], i),
            ("gemm_coll_moe_combine", [vp, i64, vp, vp, i64, i, i64, vp, i, i64, vp, vp], i),
            ("gemm_coll_lora_add", [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i, i, vp, vp, u64, vp], i)):
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
