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


# a product for each way to run one beyond the few rows, ragged in all lengths and more than eight steps of k deep
OF_EACH_PLAN = [
    ("fp16", 97, 101, 1100, (64, 64, 1)), ("bf16", 301, 397, 4111, (64, 64, 9)), ("bf16", 1501, 2051, 1101, (128, 64, 1)),
    ("fp16", 2637, 208, 8305, (128, 64, 6)), ("fp16", 2051, 2053, 1111, (128, 128, 1)),
    ("bf16", 517, 2053, 8305, (128, 128, 3)), ("fp16", 3005, 4103, 1105, (256, 256, 1)),
    ("fp32", 301, 391, 1101, (64, 64, 1)), ("fp32", 301, 397, 4111, (64, 64, 9)), ("fp32", 1503, 1505, 1101, (128, 64, 1)),
    ("fp32", 1803, 515, 3001, (128, 64, 3)), ("fp32", 2051, 2053, 1111, (128, 128, 1)),
    ("fp32", 517, 2053, 6001, (128, 128, 3)), ("fp32", 3005, 5003, 1105, (256, 256, 1)),
]
