"""Python binding of libiris_local.so: one GPU's share of Iris-style fused
communication + GEMM ops on MI355X (gfx950).

Argument marshalling only: every step of every op runs in the library's HIP
kernels. PyTorch supplies device memory (tensors) and the stream. The
functions carry the names of the C entry points declared in
include/iris_local.h, which states each operation, its source on the pages,
argument layouts, ownership and error behaviour:

  iris_ag_mm          all_gather(A shards along K) -> gathered buffer; C = gathered @ B + bias
  iris_mm_rs_local    C = A @ B + bias; out = C[:, rank slice] + sum(partials)
  iris_mm_ar_local    C = A @ B + bias; out = C + sum(partials)
  iris_concurrent     C = A @ B + bias beside an independent all_reduce of W buffers

and, in block-scaled 8-bit floating point (Fp8: codes, scales):

  iris_fp8_quantize    a matrix to 8 bits, along its rows and / or transposed
  iris_fp8_mm          C = A @ B^T + bias
  iris_fp8_swiglu      h = silu(gate) * up, gate and up kept in 8 bits if wanted
  iris_fp8_swiglu_bwd  its backward pass from the kept gate and up

There is no fallback: if the library is missing or fails to load, importing
this package raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, fields
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libiris_local.so")

IRIS_MAX_W = 16
IRIS_MODE_FUSED = 0
IRIS_MODE_SEQUENTIAL = 1
IRIS_MODE_TWO_STREAM = 2
IRIS_FLAG_NO_STEAL = 1
IRIS_FLAG_BIAS_ALONG_M = 2
IRIS_FLAG_NO_LOCKSTEP = 4
IRIS_FLAG_ACCUMULATE = 8
IRIS_OP_AG_MM = 1
IRIS_OP_MM_RS = 2
IRIS_OP_MM_AR = 3
IRIS_OP_CONCURRENT = 4
IRIS_OP_MM_AG = 5
IRIS_COLL_ALL_REDUCE = 1
IRIS_COLL_ALL_GATHER = 2
IRIS_COLL_REDUCE_SCATTER = 3
IRIS_COLL_ALL_TO_ALL = 4
IRIS_COLL_BROADCAST = 5

STATUS = {
    0: "IRIS_OK", 1: "IRIS_ERR_INVALID_ARG", 2: "IRIS_ERR_UNSUPPORTED", 3: "IRIS_ERR_CONFIG",
    4: "IRIS_ERR_ALIGNMENT", 5: "IRIS_ERR_NO_MEMORY", 6: "IRIS_ERR_HIP", 7: "IRIS_ERR_WORKSPACE",
    8: "IRIS_ERR_NO_DEVICE", 9: "IRIS_ERR_DEVICE_TIMEOUT",
}


class IrisError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class _Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "block_m", "block_n", "block_k", "group_m", "gemm_wgs", "comm_block_m", "comm_block_n", "comm_chunk",
        "mode", "flags")]


@dataclass
class Config:
    """iris_config_t; a field <= 0 means automatic (tuned cache, else default)."""
    block_m: int = 0
    block_n: int = 0
    block_k: int = 0
    group_m: int = 0
    gemm_wgs: int = 0
    comm_block_m: int = 0
    comm_block_n: int = 0
    comm_chunk: int = 0
    mode: int = IRIS_MODE_FUSED
    flags: int = 0

    def _c(self) -> _Config:
        return _Config(*[int(getattr(self, f.name)) for f in fields(self)])


class _OpArgs(ctypes.Structure):
    _fields_ = [
        ("op", ctypes.c_int32), ("C", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("A", ctypes.c_void_p), ("srcs", ctypes.POINTER(ctypes.c_void_p)),
        ("W", ctypes.c_int32), ("rank", ctypes.c_int32), ("collective", ctypes.c_int32), ("B", ctypes.c_void_p),
        ("bias", ctypes.c_void_p), ("M", ctypes.c_int64), ("N", ctypes.c_int64),
        ("K", ctypes.c_int64), ("comm_elems", ctypes.c_int64), ("cfg", _Config),
    ]


class _Fp8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("ld_scales", ctypes.c_int64), ("block", ctypes.c_int32)]


class _PredictParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in (
        "gemm_tflops_per_cu", "tile_overhead_us", "comm_gbps_per_cu", "comm_gbps_chip", "unit_overhead_us",
        "gemm_tflops_per_cu_max", "gemm_slowdown", "comm_slowdown", "phase_penalty")]


class _DeviceInfo(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int32), ("compute_units", ctypes.c_int32),
                ("clock_khz", ctypes.c_int32), ("memory_clock_khz", ctypes.c_int32),
                ("lds_bytes_per_cu", ctypes.c_int32), ("global_mem_bytes", ctypes.c_int64),
                ("arch", ctypes.c_char * 64), ("peak_fp16_tflops", ctypes.c_double),
                ("peak_hbm_gbps", ctypes.c_double)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                          f"python gemm_collective_tile_amd/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    vpp = ctypes.POINTER(ctypes.c_void_p)
    cfgp = ctypes.POINTER(_Config)
    f8 = ctypes.POINTER(_Fp8)
    sig = {
        "iris_ag_mm": [vp, vp, vpp, i32, vp, vp, i64, i64, i64, cfgp, vp, sz, vp],
        "iris_ag_mm_noalloc": [vp, vp, vpp, i32, vp, vp, i64, i64, i64, cfgp, vp],
        "iris_mm_rs_local": [vp, vp, vp, vp, vp, vpp, i32, i32, i64, i64, i64, cfgp, vp, sz, vp],
        "iris_mm_ar_local": [vp, vp, vp, vp, vp, vpp, i32, i64, i64, i64, cfgp, vp, sz, vp],
        "iris_concurrent": [vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, vpp, i32, i64, cfgp, vp, sz, vp],
        "iris_mm_ag_local": [vp, vp, vp, vp, vpp, i32, i32, i64, i64, i64, cfgp, vp, sz, vp],
        "iris_fp8_quantize": [f8, f8, vp, i32, i64, f8, i64, i64, vp],
        "iris_fp8_mm": [vp, i32, i64, f8, f8, vp, i64, i64, i64, i32, vp, sz, vp],
        "iris_fp8_swiglu": [f8, f8, f8, vp, vp, i32, i64, i64, i64, i64, vp],
        "iris_fp8_swiglu_bwd": [f8, f8, f8, f8, f8, vp, i32, i64, f8, f8, i64, i64, vp],
        "iris_grid_size": [ctypes.c_int32, cfgp],
        "iris_tune_gemm_wgs": [ctypes.POINTER(_OpArgs), ctypes.POINTER(i32), i32, i32, i32,
                               ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_float), vp],
        "iris_predict_gemm_wgs": [ctypes.POINTER(_OpArgs), i32, ctypes.POINTER(i32), i32,
                                  ctypes.POINTER(_PredictParams), ctypes.POINTER(ctypes.c_float),
                                  ctypes.POINTER(i32)],
        "iris_last_windows": [vp, vp] + [ctypes.POINTER(ctypes.c_double)] * 4,
        "iris_check_device_error": [vp, vp],
        "iris_last_clock": [vp, vp, ctypes.POINTER(ctypes.c_double)],
        "iris_mfma_ceiling": [i32, i32, vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)],
        "iris_device_info": [i32, ctypes.POINTER(_DeviceInfo)],
        "iris_status_str": [i32],
        "iris_last_error_message": [],
        "iris_finalize": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.iris_workspace_size.argtypes = [i32, i64, i64, i64, i32, cfgp]
    lib.iris_workspace_size.restype = sz
    lib.iris_fp8_mm_workspace_size.argtypes = [i64, i64, i64]
    lib.iris_fp8_mm_workspace_size.restype = sz
    lib.iris_status_str.restype = ctypes.c_char_p
    lib.iris_last_error_message.restype = ctypes.c_char_p
    return lib


_lib = _load()


# --------------------------------------------------------------- marshalling

def _check(status: int) -> None:
    if status != 0:
        raise IrisError(status, _lib.iris_last_error_message().decode())


def _ptr(t: Optional[torch.Tensor], name: str, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float16:
        raise TypeError(f"{name} must be a float16 torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    return ctypes.c_void_p(t.data_ptr())


def _ptr_array(ts: Sequence[torch.Tensor], name: str):
    arr = (ctypes.c_void_p * max(1, len(ts)))()
    for i, t in enumerate(ts):
        arr[i] = _ptr(t, f"{name}[{i}]").value
    return arr


def _cfg(config) -> Optional[ctypes.pointer]:
    if config is None:
        return None
    if isinstance(config, dict):
        config = Config(**config)
    return ctypes.pointer(config._c())


# The current stream's handle; building the torch.cuda.Stream object around it
# costs 3 us a call on the host.
_current_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream(stream):
    if stream is None:
        return _current_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ws(workspace: Optional[torch.Tensor]):
    if workspace is None:
        return None, 0
    return ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()


def _shape2(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


# Shape checks. They run before any pointer is taken: a tensor whose shape
# does not match the M, N, K, W the library derives would be read or written
# past its end by the kernels.

def _want_shape(t, shape, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _want_numel(t, n: int, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")


def _want_count(ts, n: int, name: str) -> None:
    if len(ts) != n:
        raise ValueError(f"{name} holds {len(ts)} tensors, expected {n}")


def _flags(config) -> int:
    if config is None:
        return 0
    return int(config.get("flags", 0) if isinstance(config, dict) else config.flags)


def _bias_along_m(config) -> bool:
    return bool(_flags(config) & IRIS_FLAG_BIAS_ALONG_M)


def _want_bias(bias, M: int, N: int, config) -> None:
    if bias is not None:
        _want_numel(bias, M if _bias_along_m(config) else N, "bias")


def _want_w(W: int) -> None:
    if not 1 <= int(W) <= IRIS_MAX_W:
        raise ValueError(f"W must be in [1, {IRIS_MAX_W}] (got {W})")


def _validate(op, config, C=None, out=None, A=None, srcs=(), W=1, B=None, bias=None, M=0, N=0, K=0,
              comm_elems=0, collective=IRIS_COLL_ALL_REDUCE):
    """Checks every tensor of op `op` against the shape the library derives
    (K is K_local for all_gather_matmul)."""
    _want_w(W)
    if op == IRIS_OP_AG_MM:
        _want_count(srcs, W, "A_shards")
        for s, t in enumerate(srcs):
            _want_shape(t, (M, K), f"A_shards[{s}]")
        _want_shape(B, (W * K, N), "B")
        _want_shape(C, (M, N), "C")
        _want_shape(out, (M, W * K), "A_gathered")
    elif op in (IRIS_OP_MM_RS, IRIS_OP_MM_AR):
        if op == IRIS_OP_MM_RS and N % W != 0:
            raise ValueError(f"N ({N}) must be divisible by W ({W})")
        cols = N // W if op == IRIS_OP_MM_RS else N
        _want_shape(A, (M, K), "A")
        _want_shape(B, (K, N), "B")
        _want_shape(C, (M, N), "C")
        _want_shape(out, (M, cols), "out")
        _want_count(srcs, W - 1, "partials")
        for p, t in enumerate(srcs):
            _want_shape(t, (M, cols), f"partials[{p}]")
    elif op == IRIS_OP_CONCURRENT:
        _want_shape(A, (M, K), "A")
        _want_shape(B, (K, N), "B")
        _want_shape(C, (M, N), "C")
        _want_count(srcs, W, "comm_in")
        for w, t in enumerate(srcs):
            _want_numel(t, comm_elems, f"comm_in[{w}]")
        if collective in _COMM_OUT_LEN:
            _want_numel(out, _COMM_OUT_LEN[collective](comm_elems, W), "comm_out")
    elif op == IRIS_OP_MM_AG:
        _want_shape(A, (M, K), "A")
        _want_shape(B, (K, N), "B")
        _want_shape(out, (M * W, N), "out")
        _want_count(srcs, W - 1, "peers")
        for p, t in enumerate(srcs):
            _want_shape(t, (M, N), f"peers[{p}]")
    else:
        raise ValueError(f"unknown op {op}")
    _want_bias(bias, M, N, config)


_COMM_OUT_LEN = {
    IRIS_COLL_ALL_REDUCE: lambda n, W: n, IRIS_COLL_ALL_GATHER: lambda n, W: W * n,
    IRIS_COLL_REDUCE_SCATTER: lambda n, W: n // W, IRIS_COLL_ALL_TO_ALL: lambda n, W: n,
    IRIS_COLL_BROADCAST: lambda n, W: n,
}


# ----------------------------------------------------------------------- ops

def iris_ag_mm(C, A_gathered, A_shards, B, bias=None, config=None, workspace=None, stream=None):
    """all_gather_matmul local share: A_gathered = concat_K(A_shards); C = A_gathered @ B + bias."""
    W = len(A_shards)
    if W < 1:
        raise ValueError("A_shards is empty")
    M, K_local = _shape2(A_shards[0], "A_shards[0]")
    N = _shape2(B, "B")[1]
    _validate(IRIS_OP_AG_MM, config, C=C, out=A_gathered, srcs=A_shards, W=W, B=B, bias=bias, M=M, N=N,
              K=K_local)
    ws, wsb = _ws(workspace)
    _check(_lib.iris_ag_mm(_ptr(C, "C"), _ptr(A_gathered, "A_gathered"), _ptr_array(A_shards, "A_shards"),
                           W, _ptr(B, "B"), _ptr(bias, "bias", True), M, N, K_local, _cfg(config),
                           ws, wsb, _stream(stream)))


def iris_ag_mm_noalloc(C, A_gathered, A_shards, B, bias=None, config=None, stream=None):
    """iris_ag_mm on the library's static device scratch (no workspace, no
    allocation); calls that overlap in time on one GPU race."""
    W = len(A_shards)
    if W < 1:
        raise ValueError("A_shards is empty")
    M, K_local = _shape2(A_shards[0], "A_shards[0]")
    N = _shape2(B, "B")[1]
    _validate(IRIS_OP_AG_MM, config, C=C, out=A_gathered, srcs=A_shards, W=W, B=B, bias=bias, M=M, N=N,
              K=K_local)
    _check(_lib.iris_ag_mm_noalloc(_ptr(C, "C"), _ptr(A_gathered, "A_gathered"),
                                   _ptr_array(A_shards, "A_shards"), W, _ptr(B, "B"), _ptr(bias, "bias", True),
                                   M, N, K_local, _cfg(config), _stream(stream)))


def iris_mm_rs_local(out, C, A, B, partials, W, rank=0, bias=None, config=None, workspace=None,
                     stream=None):
    """matmul_reduce_scatter local share: C = A @ B + bias; out = C[:, rank*N/W:(rank+1)*N/W] + sum(partials)."""
    M, K = _shape2(A, "A")
    N = _shape2(B, "B")[1]
    _validate(IRIS_OP_MM_RS, config, C=C, out=out, A=A, srcs=partials, W=W, B=B, bias=bias, M=M, N=N, K=K)
    ws, wsb = _ws(workspace)
    _check(_lib.iris_mm_rs_local(_ptr(out, "out"), _ptr(C, "C"), _ptr(A, "A"), _ptr(B, "B"),
                                 _ptr(bias, "bias", True), _ptr_array(partials, "partials"), W, rank,
                                 M, N, K, _cfg(config), ws, wsb, _stream(stream)))


def iris_mm_ar_local(out, C, A, B, partials, W, bias=None, config=None, workspace=None, stream=None):
    """matmul_all_reduce local share: C = A @ B + bias; out = C + sum(partials)."""
    M, K = _shape2(A, "A")
    N = _shape2(B, "B")[1]
    _validate(IRIS_OP_MM_AR, config, C=C, out=out, A=A, srcs=partials, W=W, B=B, bias=bias, M=M, N=N, K=K)
    ws, wsb = _ws(workspace)
    _check(_lib.iris_mm_ar_local(_ptr(out, "out"), _ptr(C, "C"), _ptr(A, "A"), _ptr(B, "B"),
                                 _ptr(bias, "bias", True), _ptr_array(partials, "partials"), W,
                                 M, N, K, _cfg(config), ws, wsb, _stream(stream)))


def iris_concurrent(C, A, B, comm_out, comm_in, bias=None, collective=IRIS_COLL_ALL_REDUCE, rank=0,
                    config=None, workspace=None, stream=None):
    """C = A @ B + bias, and independently the local share of `collective`
    over the W buffers comm_in (every rank's buffer, own included) into
    comm_out; `rank` is this rank (the root for broadcast)."""
    M, K = _shape2(A, "A")
    N = _shape2(B, "B")[1]
    W = len(comm_in)
    if W < 1:
        raise ValueError("comm_in is empty")
    n = comm_in[0].numel()
    _validate(IRIS_OP_CONCURRENT, config, C=C, out=comm_out, A=A, srcs=comm_in, W=W, B=B, bias=bias, M=M, N=N,
              K=K, comm_elems=n, collective=collective)
    ws, wsb = _ws(workspace)
    _check(_lib.iris_concurrent(_ptr(C, "C"), _ptr(A, "A"), _ptr(B, "B"), _ptr(bias, "bias", True),
                                M, N, K, collective, rank, _ptr(comm_out, "comm_out"),
                                _ptr_array(comm_in, "comm_in"), W, n, _cfg(config),
                                ws, wsb, _stream(stream)))


def iris_mm_ag_local(out, A, B, peers, W, rank=0, bias=None, config=None, workspace=None, stream=None):
    """matmul_all_gather local share: out (M*W, N) holds every rank's A @ B + bias
    along M; this rank's block is computed, the W-1 `peers` (M, N) are copied."""
    M, K = _shape2(A, "A")
    N = _shape2(B, "B")[1]
    _validate(IRIS_OP_MM_AG, config, out=out, A=A, srcs=peers, W=W, B=B, bias=bias, M=M, N=N, K=K)
    ws, wsb = _ws(workspace)
    _check(_lib.iris_mm_ag_local(_ptr(out, "out"), _ptr(A, "A"), _ptr(B, "B"), _ptr(bias, "bias", True),
                                 _ptr_array(peers, "peers"), W, rank, M, N, K, _cfg(config), ws, wsb,
                                 _stream(stream)))


# ---------------------------------------------------------- 8-bit operators

_FP8_TYPES = {torch.float16: 1, torch.bfloat16: 2, torch.float32: 3}


class Fp8:
    """A block-scaled 8-bit matrix: `codes` (rows, cols) float8_e4m3fn or uint8,
    `scales` (ceil(rows / block), ceil(cols / 128)) float8_e8m0fnu or uint8,
    `block` 1 (a scale for every 1 x 128 entries) or 128 (128 x 128). An entry's
    value is its code times 2^(scale byte - 127). Rows of codes start at
    multiples of 16 bytes and, in an operand of iris_fp8_mm, rows of scales at
    multiples of 4; the last row is followed by memory up to the next such
    multiple (iris_fp8_empty lays memory out that way).

    The object is a handle: it reads the tensors' addresses once and holds the
    tensors, so their memory must not be exchanged (set_, resize_) under it.
    """
    __slots__ = ("codes", "scales", "block", "shape", "_c", "_p", "_device", "_scale_words")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, block: int = 1):
        rows, cols = _shape2(codes, "codes")
        if codes.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError("codes must be a float8_e4m3fn (or uint8) torch tensor")
        if not isinstance(scales, torch.Tensor) or scales.dtype not in (torch.float8_e8m0fnu, torch.uint8):
            raise TypeError("scales must be a float8_e8m0fnu (or uint8) torch tensor")
        if block not in (1, 128):
            raise ValueError(f"block must be 1 or 128 (got {block})")
        _want_shape(scales, (-(-rows // block), -(-cols // 128)), "scales")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        for t, name in ((codes, "codes"), (scales, "scales")):
            if t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1:
                raise ValueError(f"{name} must be contiguous along its rows")
        ld, lds = _pitch(codes, 16), _pitch(scales, 4)
        if codes.numel() > 0:
            if ld % 16 != 0:
                raise ValueError(f"rows of codes must start at multiples of 16 bytes (pitch {ld}); see iris_fp8_empty")
            end = codes.storage_offset() + (rows - 1) * ld + -(-cols // 16) * 16
            if end > codes.untyped_storage().nbytes():
                raise ValueError("the last row of codes must be followed by memory up to the next multiple of 16 bytes")
        # whether the scales can be read in words of four, as products do
        end = scales.storage_offset() + (scales.shape[0] - 1) * lds + -(-scales.shape[1] // 4) * 4
        self._scale_words = scales.numel() == 0 or end <= scales.untyped_storage().nbytes()
        self.codes, self.scales, self.block, self.shape = codes, scales, block, (rows, cols)
        self._device = codes.get_device()   # -1: not on a GPU
        self._c = _Fp8(codes.data_ptr(), scales.data_ptr(), ld, lds, block)
        self._p = ctypes.pointer(self._c)


def _pitch(t: torch.Tensor, unit: int) -> int:
    """Row pitch in elements; a single row has any pitch, so it gets a whole one."""
    return t.stride(0) if t.shape[0] > 1 else -(-max(1, t.shape[1]) // unit) * unit


def iris_fp8_empty(rows: int, cols: int, block: int = 1, device=None) -> Fp8:
    """Memory of a (rows, cols) block-scaled matrix, laid out as every 8-bit
    operator takes it: codes with a row pitch that is a multiple of 16 (of 128
    beyond 512 columns), scales with one that is a multiple of 4 (uninitialised).

    Rows in whole 128-byte lines cost little memory there and save a product
    the second line of every piece it loads: 2048 x 1984 x 2640 takes 21.7 us with
    a pitch of 2688 and 27.3 with 2640, 8192 x 8192 x 8000 437 with 8192 and 466
    with 8000."""
    device = torch.device("cuda") if device is None else device
    nb = -(-cols // 128)
    unit = 128 if cols > 512 else 16
    codes = torch.empty((rows, -(-cols // unit) * unit), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    scales = torch.empty((-(-rows // block), -(-nb // 4) * 4), dtype=torch.uint8, device=device)
    return Fp8(codes[:, :cols], scales.view(torch.float8_e8m0fnu)[:, :nb], block)


# These run once per call in front of a 2 us launch, so they do little more than
# the comparisons themselves. `dev` is the device that all operands have to be on:
# the current one, where the kernels run.

def _elsewhere(name: str, device: int, dev: int):
    if device < 0 or dev < 0:
        return ValueError(f"{name if device < 0 else 'every operand'} must be on a GPU")
    return ValueError(f"{name} is on GPU {device}, not on GPU {dev}")


def _fp8(q, shape, name: str, dev: int):
    """q's C struct, after the check of its kind, shape and device."""
    if q.__class__ is not Fp8:
        raise TypeError(f"{name} must be an Fp8 matrix") if q is not None else ValueError(f"{name} is required")
    if q.shape != shape:
        raise ValueError(f"{name} has shape {q.shape}, expected {shape}")
    if q._device != dev or dev < 0:
        raise _elsewhere(name, q._device, dev)
    return q._p


def _plain(t, name: str, kinds, rows: int, cols: int, dev: int):
    """(pointer, type, row pitch) of a row-major matrix with any row pitch."""
    kind = kinds.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be one of {', '.join(str(d)[6:] for d in kinds)}")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    device = t.get_device()
    if device != dev or dev < 0:
        raise _elsewhere(name, device, dev)
    return t.data_ptr(), kind, (ld if rows > 1 else cols)


def _fp8_stream(stream, dev: int):
    """The stream's handle (the current one, a torch stream or a handle), after the check of the current device."""
    current = _current_device()
    if current != dev:
        raise ValueError(f"the operands are on GPU {dev}, the current device is {current}")
    if stream is None:
        return _current_stream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise _elsewhere("stream", stream.device_index, dev)
    return _stream(stream)


def _fp8_ws(workspace, dev: int):
    """(pointer, bytes) of a caller's workspace, which the kernels write from its first byte on."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    device = workspace.get_device()
    if device != dev or dev < 0:
        raise _elsewhere("workspace", device, dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


_FP8_HALVES = {torch.float16: 1, torch.bfloat16: 2}


def iris_fp8_quantize(x, q: Optional[Fp8] = None, q_t: Optional[Fp8] = None, stream=None) -> None:
    """x (rows, cols) to 8 bits: q (rows, cols) with blocks along its rows and /
    or q_t (cols, rows), x transposed, both in one pass. x is a float16, bfloat16
    or float32 tensor, or an Fp8 matrix (then only q_t, blocks of 1 x 128)."""
    from8 = x.__class__ is Fp8
    if not from8 and (not isinstance(x, torch.Tensor) or x.dim() != 2):
        _shape2(x, "x")
    shape = rows, cols = x.shape
    dev = x._device if from8 else x.get_device()
    qp = None if q is None else _fp8(q, (rows, cols), "q", dev)
    qtp = None if q_t is None else _fp8(q_t, (cols, rows), "q_t", dev)
    if from8:
        ptr, kind, ld, x8 = None, 0, 0, _fp8(x, shape, "x", dev)
    else:
        ptr, kind, ld = _plain(x, "x", _FP8_TYPES, rows, cols, dev)
        x8 = None
    st = _lib.iris_fp8_quantize(qp, qtp, ptr, kind, ld, x8, rows, cols,
                                _current_stream(dev) if stream is None and _current_device() == dev else _fp8_stream(stream, dev))
    if st:
        _check(st)


def iris_fp8_mm(C, A: Fp8, B: Fp8, bias=None, accumulate=False, config=None, workspace=None, stream=None) -> None:
    """C = A @ B^T + bias (+ C with accumulate, or the flag in config): A (M, K) Fp8 with blocks of
    1 x 128, B (N, K) Fp8, C (M, N) float16, bfloat16 or float32, bias of C's type.
    A float32 C has exact products and 32-bit sums; a 16-bit one drops, of every 8
    products, what lies under 2^-13 of the largest."""
    if A.__class__ is not Fp8 or B.__class__ is not Fp8:
        raise TypeError("A and B must be Fp8 matrices")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError(f"B has shape {B.shape}, expected ({N}, {K})")
    if not (A._scale_words and B._scale_words):
        raise ValueError(f"the last row of {'B' if A._scale_words else 'A'}'s scales must be followed by memory up to the "
                         "next multiple of 4 bytes; see iris_fp8_empty")
    if not isinstance(C, torch.Tensor) or C.shape != (M, N):
        _want_shape(C, (M, N), "C")
    dev = A._device
    ws, wsb = (None, 0) if workspace is None else _fp8_ws(workspace, dev)
    flags = IRIS_FLAG_ACCUMULATE if accumulate else _flags(config) & IRIS_FLAG_ACCUMULATE
    bias_ptr = None
    if bias is not None:
        _want_bias(bias, M, N, config)
        if bias.dtype != C.dtype:
            raise TypeError(f"bias must be {C.dtype} as C is")
        if not bias.is_contiguous():
            raise ValueError("bias must be contiguous")
        if _bias_along_m(config):
            flags |= IRIS_FLAG_BIAS_ALONG_M
    ptr, kind, ld = _plain(C, "C", _FP8_TYPES, M, N, dev)
    if bias is not None:
        if bias.get_device() != dev:
            raise _elsewhere("bias", bias.get_device(), dev)
        bias_ptr = bias.data_ptr()
    st = _lib.iris_fp8_mm(ptr, kind, ld, _fp8(A, A.shape, "A", dev), _fp8(B, B.shape, "B", dev), bias_ptr, M, N, K, flags,
                          ws, wsb,
                          _current_stream(dev) if stream is None and _current_device() == dev else _fp8_stream(stream, dev))
    if st:
        _check(st)


def iris_fp8_swiglu(h: Fp8, gate, up, gate_kept: Optional[Fp8] = None, up_kept: Optional[Fp8] = None,
                    stream=None) -> None:
    """h = silu(gate) * up in 8 bits; gate, up (rows, cols) float16 or bfloat16
    (views of one matrix will do); gate_kept and up_kept receive them in 8 bits."""
    if not isinstance(gate, torch.Tensor) or gate.dim() != 2:
        _shape2(gate, "gate")
    shape = rows, cols = gate.shape
    if not isinstance(up, torch.Tensor) or up.shape != shape:
        _want_shape(up, shape, "up")
    if up.dtype != gate.dtype:
        raise TypeError("gate and up must have one dtype")
    dev = gate.get_device()
    hp = _fp8(h, shape, "h", dev)
    kept = gate_kept is not None or up_kept is not None
    gkp = _fp8(gate_kept, shape, "gate_kept", dev) if kept else None
    ukp = _fp8(up_kept, shape, "up_kept", dev) if kept else None
    gp, kind, gld = _plain(gate, "gate", _FP8_HALVES, rows, cols, dev)
    up_ptr, _, uld = _plain(up, "up", _FP8_HALVES, rows, cols, dev)
    st = _lib.iris_fp8_swiglu(hp, gkp, ukp, gp, up_ptr, kind, gld, uld, rows, cols,
                              _current_stream(dev) if stream is None and _current_device() == dev else _fp8_stream(stream, dev))
    if st:
        _check(st)


def iris_fp8_swiglu_bwd(dgate: Fp8, dup: Fp8, dh, gate_kept: Fp8, up_kept: Fp8, dgate_t: Optional[Fp8] = None,
                        dup_t: Optional[Fp8] = None, h_t: Optional[Fp8] = None, stream=None) -> None:
    """Backward pass of iris_fp8_swiglu at the kept gate and up: dgate, dup
    (rows, cols) and, if given, dgate_t, dup_t and the recomputed h_t (cols,
    rows), all in 8 bits; dh (rows, cols) float16 or bfloat16."""
    if not isinstance(dh, torch.Tensor) or dh.dim() != 2:
        _shape2(dh, "dh")
    shape = rows, cols = dh.shape
    turned = (cols, rows)
    dev = dh.get_device()
    st = _lib.iris_fp8_swiglu_bwd(
        _fp8(dgate, shape, "dgate", dev), _fp8(dup, shape, "dup", dev),
        None if dgate_t is None else _fp8(dgate_t, turned, "dgate_t", dev),
        None if dup_t is None else _fp8(dup_t, turned, "dup_t", dev),
        None if h_t is None else _fp8(h_t, turned, "h_t", dev),
        *_plain(dh, "dh", _FP8_HALVES, rows, cols, dev), _fp8(gate_kept, shape, "gate_kept", dev),
        _fp8(up_kept, shape, "up_kept", dev), rows, cols,
        _current_stream(dev) if stream is None and _current_device() == dev else _fp8_stream(stream, dev))
    if st:
        _check(st)


def iris_fp8_mm_workspace_size(M, N, K) -> int:
    return int(_lib.iris_fp8_mm_workspace_size(M, N, K))


# ------------------------------------------------------------------- helpers

def iris_workspace_size(op, M, N, K, W, config=None) -> int:
    return int(_lib.iris_workspace_size(op, M, N, K, W, _cfg(config)))


def iris_grid_size(config=None, op=IRIS_OP_AG_MM) -> int:
    """Workgroups of the fused persistent launch of `op` for this config."""
    g = _lib.iris_grid_size(op, _cfg(config))
    if g < 0:
        _check(-g)
    return g


def _op_args(op, config, C=None, out=None, A=None, srcs=(), W=1, rank=0, collective=0, B=None, bias=None,
             M=0, N=0, K=0, comm_elems=0):
    keep = _ptr_array(list(srcs), "srcs")
    a = _OpArgs()
    a.op = op
    a.C = _ptr(C, "C", True)
    a.out = _ptr(out, "out", True)
    a.A = _ptr(A, "A", True)
    a.srcs = ctypes.cast(keep, ctypes.POINTER(ctypes.c_void_p))
    a.W, a.rank, a.collective = W, rank, collective
    a.B = _ptr(B, "B", True)
    a.bias = _ptr(bias, "bias", True)
    a.M, a.N, a.K, a.comm_elems = M, N, K, comm_elems
    a.cfg = (config if isinstance(config, Config) else Config(**(config or {})))._c()
    return a, keep


def iris_tune_gemm_wgs(op, candidates, reps=5, config=None, stream=None, *, top_k=0, C=None, out=None, A=None,
                       srcs=(), W=1, rank=0, collective=0, B=None, bias=None, M=0, N=0, K=0, comm_elems=0):
    """Sweep gemm_wgs over `candidates` (the static default is always added),
    cache and return (best, {candidate: median ms}). With top_k > 0 only the
    top_k candidates the predictor ranks best are run (the others read -1)."""
    _validate(op, config, C=C, out=out, A=A, srcs=srcs, W=W, B=B, bias=bias, M=M, N=N, K=K,
              comm_elems=comm_elems, collective=collective or IRIS_COLL_ALL_REDUCE)
    a, keep = _op_args(op, config, C, out, A, srcs, W, rank, collective, B, bias, M, N, K, comm_elems)
    cands = (ctypes.c_int32 * max(1, len(candidates)))(*candidates)
    ms = (ctypes.c_float * max(1, len(candidates)))()
    best = ctypes.c_int32(0)
    _check(_lib.iris_tune_gemm_wgs(ctypes.byref(a), cands, len(candidates), reps, top_k, ctypes.byref(best),
                                   ms, _stream(stream)))
    del keep
    return best.value, {c: ms[i] for i, c in enumerate(candidates)}


def iris_predict_gemm_wgs(op, candidates, grid, config=None, params=None, *, W=1, rank=0, collective=0,
                          M=0, N=0, K=0, comm_elems=0):
    """Predicted makespan (ms) of the fused schedule for each gemm_wgs
    candidate on a grid of `grid` workgroups; returns (best, {candidate: ms}).
    Host only: needs the shapes, no tensors. `params` is a dict of the
    model's constants (gemm_tflops_per_cu, tile_overhead_us, comm_gbps_per_cu,
    comm_gbps_chip, unit_overhead_us, gemm_tflops_per_cu_max, gemm_slowdown,
    comm_slowdown, phase_penalty); missing ones take the defaults."""
    a, keep = _op_args(op, config, W=W, rank=rank, collective=collective, M=M, N=N, K=K, comm_elems=comm_elems)
    pp = _PredictParams(*[-1.0] * len(_PredictParams._fields_))
    for k, v in (params or {}).items():
        if k not in dict(_PredictParams._fields_):
            raise ValueError(f"unknown predictor parameter {k!r}")
        setattr(pp, k, float(v))
    cands = (ctypes.c_int32 * max(1, len(candidates)))(*candidates)
    ms = (ctypes.c_float * max(1, len(candidates)))()
    best = ctypes.c_int32(0)
    _check(_lib.iris_predict_gemm_wgs(ctypes.byref(a), grid, cands, len(candidates), ctypes.byref(pp), ms,
                                      ctypes.byref(best)))
    del keep
    return best.value, {c: ms[i] for i, c in enumerate(candidates)}


def iris_last_windows(workspace=None, stream=None):
    """(gemm_start, gemm_end, comm_start, comm_end) in ns of the last fused launch; -1 if none."""
    vals = [ctypes.c_double() for _ in range(4)]
    ws, _ = _ws(workspace)
    _check(_lib.iris_last_windows(ws, _stream(stream), *[ctypes.byref(v) for v in vals]))
    return tuple(v.value for v in vals)


def iris_last_clock(workspace=None, stream=None) -> float:
    """Shader clock (MHz) held during the last persistent launch on this
    workspace (-1 if none was recorded)."""
    v = ctypes.c_double()
    ws, _ = _ws(workspace)
    _check(_lib.iris_last_clock(ws, _stream(stream), ctypes.byref(v)))
    return v.value


def iris_mfma_ceiling(random_operands: bool = True, iters: int = 400000, stream=None):
    """(TFLOP/s, MHz): the dense fp16 MFMA rate of the current GPU with no
    memory traffic, operands random (switching as on GEMM data) or constant,
    and the shader clock it held. Waits for the run."""
    t, m = ctypes.c_double(), ctypes.c_double()
    _check(_lib.iris_mfma_ceiling(1 if random_operands else 0, int(iters), _stream(stream), ctypes.byref(t),
                                  ctypes.byref(m)))
    return t.value, m.value


def iris_check_device_error(workspace=None, stream=None) -> None:
    """Waits for the stream; raises IrisError (IRIS_ERR_DEVICE_TIMEOUT) if a
    device-side wait of a fused op on this workspace gave up since the last
    check (the outputs of those ops are then not to be trusted)."""
    ws, _ = _ws(workspace)
    _check(_lib.iris_check_device_error(ws, _stream(stream)))


def iris_device_info(device: int = 0) -> dict:
    info = _DeviceInfo()
    _check(_lib.iris_device_info(device, ctypes.byref(info)))
    return {f[0]: (getattr(info, f[0]).decode() if f[0] == "arch" else getattr(info, f[0]))
            for f in _DeviceInfo._fields_}


def iris_finalize() -> None:
    _check(_lib.iris_finalize())


def library_path() -> str:
    return LIB_PATH
