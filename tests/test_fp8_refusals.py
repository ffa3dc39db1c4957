"""What the 8-bit operators refuse, before any GPU call: the binding's checks
(TypeError, ValueError) on CPU tensors, the library's status codes on
placeholder pointers that are never read."""
import ctypes

import pytest
import torch

import gemm_collective_tile_amd as il
from gemm_collective_tile_amd import _Fp8, _lib

P, ODD = 0x100000, 0x100008


def empty(rows, cols, block=1):
    return il.iris_fp8_empty(rows, cols, block, device="cpu")


# ------------------------------------------------------------------- binding

def test_fp8_handle_refuses():
    codes, scales = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    il.Fp8(codes, scales)
    il.Fp8(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu))
    for bad in ((codes.float(), scales, 1), (codes, scales.float(), 1), (codes.to(torch.int8), scales, 1)):
        with pytest.raises(TypeError):
            il.Fp8(*bad)
    for bad in ((codes, scales[:, :1], 1), (codes, scales[:2], 1), (codes, scales, 64), (codes, scales, 128),
                (codes.reshape(2, 2, 256), scales, 1), (codes.t(), scales, 1), (codes[:, :40].contiguous()[:, :37], scales[:, :1], 1)):
        with pytest.raises(ValueError):
            il.Fp8(*bad)
    tight = torch.zeros(16 * 3 + 5, dtype=torch.uint8).as_strided((4, 5), (16, 1))
    with pytest.raises(ValueError, match="next multiple of 16"):
        il.Fp8(tight, torch.zeros((4, 1), dtype=torch.uint8))


def test_empty_gives_long_rows_whole_lines():
    assert empty(3, 513).codes.stride() == (640, 1) and empty(3, 512).codes.stride() == (512, 1)
    assert empty(2, 4095).codes.stride() == (4096, 1) and empty(2, 511).codes.stride() == (512, 1)


def test_empty_lays_rows_out():
    q = empty(5, 130, 128)
    assert q.codes.stride() == (144, 1) and q.scales.shape == (1, 2) and q.scales.dtype == torch.float8_e8m0fnu
    assert empty(300, 1000).scales.stride() == (8, 1)
    for rows, cols in ((0, 9), (9, 0), (0, 0)):
        assert empty(rows, cols).shape == (rows, cols)


def expect(kind, text, fn, *args, **kw):
    with pytest.raises(kind, match=text):
        fn(*args, **kw)


def test_quantize_refuses():
    x = torch.zeros((6, 200), dtype=torch.float16)
    f = il.iris_fp8_quantize
    expect(ValueError, "expected", f, x, empty(6, 201))
    expect(ValueError, "expected", f, x, None, empty(6, 200))
    expect(TypeError, "Fp8", f, x, torch.zeros((6, 200), dtype=torch.uint8))
    expect(ValueError, "2-D", f, x[0], empty(6, 200))
    expect(ValueError, "on a GPU", f, x, empty(6, 200))
    expect(TypeError, "must be one of", _on_gpu_checks, f, x.double())
    expect(ValueError, "contiguous along", _on_gpu_checks, f, torch.zeros((200, 6), dtype=torch.float16).t())


def _on_gpu_checks(f, x):
    f(x)      # no outputs: the plain matrix's own checks come first


def test_mm_refuses():
    A, B, C = empty(6, 200), empty(9, 200), torch.zeros((6, 9), dtype=torch.float16)
    f = il.iris_fp8_mm
    expect(ValueError, "B has shape", f, C, A, empty(9, 199))
    expect(ValueError, "C has shape", f, C[:, :8], A, B)
    expect(TypeError, "Fp8", f, C, torch.zeros(6, 200), B)
    expect(ValueError, "bias has", f, C, A, B, torch.zeros(8, dtype=torch.float16))
    expect(TypeError, "bias must be", f, C, A, B, torch.zeros(9))
    expect(ValueError, "bias has", f, C, A, B, torch.zeros(9, dtype=torch.float16),
           config=il.Config(flags=il.IRIS_FLAG_BIAS_ALONG_M))
    expect(TypeError, "C must be one of", f, C.double(), A, B)
    expect(ValueError, "contiguous along", f, torch.zeros((9, 6)).t(), A, B)
    expect(ValueError, "on a GPU", f, C, A, B)


def test_mm_refuses_scales_that_end_inside_a_word():
    """Products read a row's scales four at a time: the last row needs memory up to the next multiple of 4."""
    codes, C = torch.zeros((1, 304), dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.float16)
    whole = empty(1, 300)
    tight = il.Fp8(codes[:, :300], torch.zeros((1, 3), dtype=torch.uint8))
    pitched = torch.zeros(8 + 5, dtype=torch.uint8).as_strided((2, 5), (8, 1))
    weight = il.Fp8(torch.zeros((129, 640), dtype=torch.uint8), pitched, 128)
    late = il.Fp8(codes[:, :300], torch.zeros(8, dtype=torch.uint8)[5:].reshape(1, 3))
    for A, B, name in ((tight, whole, "A"), (whole, tight, "B"), (late, whole, "A"), (empty(1, 640), weight, "B")):
        expect(ValueError, f"{name}'s scales", il.iris_fp8_mm, torch.zeros((1, B.shape[0]), dtype=torch.float16), A, B)
    roomy = il.Fp8(codes[:, :300], torch.zeros((1, 4), dtype=torch.uint8)[:, :3])
    expect(ValueError, "on a GPU", il.iris_fp8_mm, C, roomy, whole)
    expect(ValueError, "on a GPU", il.iris_fp8_mm, C, il.Fp8(codes[:, :0], torch.zeros((1, 0), dtype=torch.uint8)), empty(1, 0))


def test_mm_refuses_workspaces():
    A, B, C = empty(100, 200), empty(90, 200), torch.zeros((100, 90), dtype=torch.float16)
    f = il.iris_fp8_mm
    expect(ValueError, "workspace must be on a GPU", f, C, A, B, workspace=torch.zeros(1 << 20))
    expect(ValueError, "workspace must be contiguous", f, C, A, B, workspace=torch.zeros(1 << 20)[::2])
    expect(TypeError, "workspace must be a torch tensor", f, C, A, B, workspace=1 << 20)


def test_swiglu_refuses():
    g, h = torch.zeros((6, 200), dtype=torch.float16), empty(6, 200)
    f = il.iris_fp8_swiglu
    expect(ValueError, "up has shape", f, h, g, g[:, :199])
    expect(TypeError, "one dtype", f, h, g, g.bfloat16())
    expect(ValueError, "h has shape", f, empty(6, 199), g, g)
    expect(ValueError, "on a GPU", f, h, g, g, h)
    b = il.iris_fp8_swiglu_bwd
    expect(ValueError, "dgate has shape", b, empty(6, 199), h, g, h, h)
    expect(ValueError, "on a GPU", b, h, h, g, h, h)
    expect(ValueError, "is required", b, None, h, g, h, h)


class OnGpu1:
    """A matrix on the second GPU, as far as the binding looks before it takes its address."""
    def __init__(self, t):
        self.dtype, self.stride = t.dtype, t.stride

    def get_device(self):
        return 1

    def data_ptr(self):
        raise AssertionError("its address was taken")


def test_operands_on_another_device_are_refused(monkeypatch):
    """The kernels run on the current device, on its stream: operands of another one would be reached over the
    link, or not at all, and ordered by no stream."""
    here, there = empty(6, 200), empty(6, 200)
    here._device, there._device = 0, 1
    assert il._fp8(here, (6, 200), "q", 0) is here._p
    expect(ValueError, "q is on GPU 1, not on GPU 0", il._fp8, there, (6, 200), "q", 0)
    expect(ValueError, "q must be on a GPU", il._fp8, empty(6, 200), (6, 200), "q", 0)
    expect(ValueError, "q must be on a GPU", il._fp8, empty(6, 200), (6, 200), "q", -1)
    expect(ValueError, "every operand must be on a GPU", il._fp8, here, (6, 200), "q", -1)
    x = torch.zeros((6, 200), dtype=torch.float16)
    expect(ValueError, "x is on GPU 1, not on GPU 0", il._plain, OnGpu1(x), "x", il._FP8_TYPES, 6, 200, 0)
    expect(ValueError, "x must be on a GPU", il._plain, x, "x", il._FP8_TYPES, 6, 200, 0)
    expect(ValueError, "q_t is on GPU 1, not on GPU 0", il.iris_fp8_quantize, here, None, turned(1))
    monkeypatch.setattr(il, "_current_device", lambda: 1)
    expect(ValueError, "operands are on GPU 0, the current device is 1", il.iris_fp8_quantize, here, None, turned(0))
    monkeypatch.setattr(il, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "Stream", type("Stream", (), {"device_index": 1, "cuda_stream": 0}))
    expect(ValueError, "stream is on GPU 1, not on GPU 0", il._fp8_stream, torch.cuda.Stream(), 0)


def turned(device):
    q = empty(200, 6)
    q._device = device
    return q


# ------------------------------------------------------------------- library

def st(status):
    return il.STATUS[status]


def m8(codes=P, scales=P, ld=1024, lds=8, block=1):
    return ctypes.pointer(_Fp8(codes, scales, ld, lds, block))


def quant(q=None, qt=None, x=P, kind=1, ldx=1024, x8=None, rows=512, cols=1000):
    return st(_lib.iris_fp8_quantize(q, qt, x, kind, ldx, x8, rows, cols, None))


def test_library_quantize_refuses():
    assert quant() == "IRIS_ERR_INVALID_ARG"                                   # no output
    assert quant(m8(), x=None) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(), kind=9) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(), ldx=999) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(), x=P + 1) == "IRIS_ERR_ALIGNMENT"
    assert quant(m8(codes=ODD)) == "IRIS_ERR_ALIGNMENT"
    assert quant(m8(ld=1023 + 9)) == "IRIS_ERR_ALIGNMENT"
    assert quant(m8(ld=992)) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(lds=7)) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(block=3)) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(codes=None)) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(), m8(block=128, ld=512)) == "IRIS_ERR_INVALID_ARG"        # two kinds of block
    assert quant(m8(), rows=-1) == "IRIS_ERR_INVALID_ARG"
    assert quant(m8(), rows=1 << 31) == "IRIS_ERR_UNSUPPORTED"
    assert quant(m8(ld=1 << 23)) == "IRIS_ERR_UNSUPPORTED"
    assert quant(m8(), ldx=1 << 23) == "IRIS_ERR_UNSUPPORTED"
    assert quant(m8(), x8=m8()) == "IRIS_ERR_INVALID_ARG"                      # x and x8
    assert quant(m8(), x=None, x8=m8()) == "IRIS_ERR_UNSUPPORTED"              # 8 bits to rows
    assert quant(None, m8(block=128, ld=512), x=None, x8=m8()) == "IRIS_ERR_UNSUPPORTED"
    assert quant(None, m8(ld=512), x=None, x8=m8(block=128)) == "IRIS_ERR_UNSUPPORTED"
    assert quant(m8(), rows=0) == "IRIS_OK" and quant(m8(), cols=0) == "IRIS_OK"


def test_library_refuses_more_tiles_than_a_launch_holds():
    """2^23 tiles of 128 x 128, 512 threads each, are 2^32 threads."""
    wide = dict(ldx=1 << 22, rows=(1 << 15) + 1, cols=1 << 22)
    assert quant(m8(ld=1 << 22, lds=1 << 15, block=128), **wide) == "IRIS_ERR_UNSUPPORTED"
    assert quant(None, m8(ld=1 << 16, lds=1 << 9), **wide) == "IRIS_ERR_UNSUPPORTED"
    assert quant(m8(block=128, ld=128), ldx=128, rows=1 << 30, cols=128) == "IRIS_ERR_UNSUPPORTED"
    big = ctypes.pointer(_Fp8(P, P, 1 << 22, 1 << 15, 1))
    assert st(_lib.iris_fp8_swiglu_bwd(big, big, None, None, None, P, 1, 1 << 22, big, big, (1 << 15) + 1, 1 << 22,
                                       None)) == "IRIS_ERR_UNSUPPORTED"
    assert mm(M=1 << 30, N=1 << 14, ldc=1 << 14) == "IRIS_ERR_UNSUPPORTED"


def mm(C=P, kind=1, ldc=512, A=None, B=None, bias=None, M=512, N=512, K=1000, flags=0, ws=None, wsb=0):
    return st(_lib.iris_fp8_mm(C, kind, ldc, A or m8(), B or m8(block=128), bias, M, N, K, flags, ws, wsb, None))


def test_library_mm_refuses():
    assert mm(C=None) == "IRIS_ERR_INVALID_ARG"
    assert mm(kind=4) == "IRIS_ERR_INVALID_ARG"
    assert mm(ldc=511) == "IRIS_ERR_INVALID_ARG"
    assert mm(C=P + 1) == "IRIS_ERR_ALIGNMENT"
    assert mm(bias=P + 1) == "IRIS_ERR_ALIGNMENT"
    assert mm(A=m8(block=128)) == "IRIS_ERR_UNSUPPORTED"
    assert mm(A=m8(scales=P + 2)) == "IRIS_ERR_ALIGNMENT"
    assert mm(B=m8(lds=10, block=128)) == "IRIS_ERR_ALIGNMENT"
    assert mm(B=m8(ld=960)) == "IRIS_ERR_INVALID_ARG"
    assert mm(flags=1) == "IRIS_ERR_CONFIG"
    assert mm(M=-1) == "IRIS_ERR_INVALID_ARG"
    assert mm(M=1 << 31) == "IRIS_ERR_UNSUPPORTED"
    assert mm(K=1 << 22, A=m8(ld=1 << 22, lds=1 << 16), B=m8(ld=1 << 22, lds=1 << 16)) == "IRIS_ERR_UNSUPPORTED"
    assert mm(M=0) == "IRIS_OK" and mm(N=0) == "IRIS_OK"
    need = il.iris_fp8_mm_workspace_size(256, 512, 11008)
    assert need > 0
    wide = dict(A=m8(ld=11008, lds=88), B=m8(ld=11008, lds=88, block=128), M=256, K=11008)
    assert mm(ws=P, wsb=0, **wide) == "IRIS_ERR_WORKSPACE"
    assert mm(ws=P + 64, wsb=need, **wide) == "IRIS_ERR_ALIGNMENT"


def test_workspace_sizes():
    f = il.iris_fp8_mm_workspace_size
    assert f(1, 4096, 4096) == 0 and f(64, 4096, 11008) == 0      # few rows: no split
    assert f(8192, 8192, 8192) == 0                               # tiles enough
    assert f(-1, 2, 3) == 0 and f(0, 0, 0) == 0
    for m in (65, 100, 129, 300, 513, 1000, 2500):
        for n in (1, 64, 130, 1376, 4096, 11008):
            for k in (0, 100, 1000, 4096, 11008, 100000):
                assert f(m, n, k) <= 512 * 128 * 128 * 4, (m, n, k)


def test_library_activation_refuses():
    def fwd(h=None, gk=None, uk=None, gate=P, up=P, kind=1, lg=1024, lu=1024, rows=512, cols=1000):
        return st(_lib.iris_fp8_swiglu(h or m8(), gk, uk, gate, up, kind, lg, lu, rows, cols, None))
    assert fwd(gk=m8()) == "IRIS_ERR_INVALID_ARG"
    assert fwd(kind=3) == "IRIS_ERR_INVALID_ARG"
    assert fwd(up=None) == "IRIS_ERR_INVALID_ARG"
    assert fwd(lg=999) == "IRIS_ERR_INVALID_ARG"
    assert fwd(h=m8(block=128)) == "IRIS_ERR_UNSUPPORTED"
    assert fwd(rows=0) == "IRIS_OK"

    def bwd(dg=None, du=None, dgt=None, dut=None, ht=None, dh=P, kind=1, ld=1024, gk=None, uk=None, rows=512, cols=1000):
        return st(_lib.iris_fp8_swiglu_bwd(dg or m8(), du or m8(), dgt, dut, ht, dh, kind, ld, gk or m8(), uk or m8(),
                                           rows, cols, None))
    assert bwd(dh=None) == "IRIS_ERR_INVALID_ARG"
    assert bwd(kind=3) == "IRIS_ERR_INVALID_ARG"
    assert bwd(dgt=m8(ld=496)) == "IRIS_ERR_INVALID_ARG"          # shorter than its 512 columns
    assert bwd(ht=m8(block=128, ld=512)) == "IRIS_ERR_UNSUPPORTED"
    assert bwd(gk=m8(codes=ODD)) == "IRIS_ERR_ALIGNMENT"
    assert bwd(cols=0) == "IRIS_OK"


def test_library_refuses_outputs_that_are_another_operand():
    """Whether an operator in place would read before it writes depends on its kernel, so none is allowed."""
    at = lambda n, ld=1024, lds=8: m8(0x1000000 * n, 0x1000000 * n + 0x800000, ld, lds)  # noqa: E731
    x, stop = 0x1000000 * 30, 7                      # operand number 7 takes the place of another below
    share = at(stop)

    def fwd(h=at(1), gk=at(2), uk=at(3), gate=x, up=x + (1 << 20)):
        return st(_lib.iris_fp8_swiglu(h, gk, uk, gate, up, 1, 1024, 1024, 512, 1000, None))
    assert fwd(gk=share, uk=share) == fwd(h=share, gk=share) == fwd(h=m8(x, P)) == "IRIS_ERR_INVALID_ARG"
    assert fwd(uk=m8(0x1000000 * 9, 0x1000000 * 2 + 0x800000)) == "IRIS_ERR_INVALID_ARG"      # scales alone

    names = ["dg", "du", "dgt", "dut", "ht", "gk", "uk"]

    def bwd(dh=x, **other):
        m = {n: at(i + 10, 512 if n.endswith("t") else 1024) for i, n in enumerate(names)}
        m.update(other)
        return st(_lib.iris_fp8_swiglu_bwd(m["dg"], m["du"], m["dgt"], m["dut"], m["ht"], dh, 1, 1024, m["gk"], m["uk"],
                                           512, 1000, None))
    for a in names[:5]:
        for b in names:
            if a != b:
                same = {n: at(stop, 512 if n.endswith("t") else 1024) for n in (a, b)}
                assert bwd(**same) == "IRIS_ERR_INVALID_ARG", (a, b)
    assert bwd(dg=m8(x, P)) == "IRIS_ERR_INVALID_ARG"
    assert quant(at(1), at(1, 512)) == quant(m8(x, P), x=x) == "IRIS_ERR_INVALID_ARG"
    assert quant(None, at(1, 512), x=None, x8=at(1)) == "IRIS_ERR_INVALID_ARG"
    assert mm(C=x, A=m8(x, P)) == mm(C=x, B=m8(x, P)) == mm(C=x, bias=x) == "IRIS_ERR_INVALID_ARG"
    assert mm(C=x, ws=x, wsb=1 << 25) == "IRIS_ERR_INVALID_ARG"
