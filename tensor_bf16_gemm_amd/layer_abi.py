"""ctypes side of include/gemm_coll_layer.h: structures and signatures.  It
needs neither torch nor the extension module, as little as the library itself."""
from __future__ import annotations

import ctypes


class Fp8Plan(ctypes.Structure):
    """Mirror of ``gc_fp8_plan`` in include/gemm_coll_layer.h."""
    _fields_ = [("tile_rows", ctypes.c_int32), ("tile_cols", ctypes.c_int32), ("splits", ctypes.c_int32)]


def declare(L: ctypes.CDLL) -> None:
    """Sets the signatures of the functions of include/gemm_coll_layer.h."""
    i, i64, vp, u64, f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_float
    for name, args in (
            ("gemm_coll_rms_norm", [vp, vp, vp, i, i64, vp, i, f, i64, i64, vp, vp, vp, vp, i64, vp]),
            ("gemm_coll_quantize_fp8", [vp, i64, i64, i, vp, vp, i64, vp]),
            ("gemm_coll_gemm_fp8", [vp, vp, i64, i64, vp, vp, i64, i64, i64, vp, i, i64, vp, vp, u64, vp]),
            ("gemm_coll_gemm_fp8_plan", [i64, i64, i64, i, i, i, ctypes.POINTER(Fp8Plan)]),
            ("gemm_coll_moe_layer", [vp, vp, i, i64, i64, i, i, i, vp, i, f, vp, vp, i, i, i64, i64, i64, vp, i,
                                     i64, vp, vp, u64, vp])):
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = i
