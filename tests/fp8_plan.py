"""How the library would run an 8-bit product, for tests: the host function behind iris_fp8_mm, no GPU."""
import ctypes

from gemm_collective_tile_amd import _lib


class Plan(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("splits", ctypes.c_int32), ("split_steps", ctypes.c_int32),
                ("ws_bytes", ctypes.c_size_t)]


_plan = _lib["_ZN4iris11fp8_mm_planElllb"]
_plan.restype, _plan.argtypes = Plan, [ctypes.c_int64] * 3 + [ctypes.c_bool]


def plan(M, N, K, dtype="fp16"):
    """(tile rows, tile columns, splits of the contraction); (0, 0, 1): the kernel for few rows."""
    p = _plan(M, N, K, dtype == "fp32")
    return (p.bm, p.bn, p.splits) if p.bm else (0, 0, 1)
