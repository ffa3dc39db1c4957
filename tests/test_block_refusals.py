"""What the block operators refuse, before any GPU call: the binding's checks (TypeError,
ValueError) on CPU tensors, the library's status codes on placeholder pointers that are
never read."""
import ctypes

import pytest
import torch

import gemm_collective_tile_amd as il
from gemm_collective_tile_amd import _Drop, _Fp8, _lib, _Norm

P, Q, R, S, ODD = 0x100000, 0x200000, 0x300000, 0x400000, 0x100001
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 4, 7


def empty(rows, cols, block=1):
    return il.iris_fp8_empty(rows, cols, block, device="cpu")


def expect(error, text, fn, *args, **kw):
    with pytest.raises(error, match=text):
        fn(*args, **kw)


# ------------------------------------------------------------------- binding

def test_dropout_handle_refuses():
    for p in (-0.1, 1.0, float("nan")):
        expect(ValueError, "in \\[0, 1\\)", il.Dropout, p, 1)
    expect(TypeError, "int64", il.Dropout, 0.1, 1, counter=torch.zeros(1))
    expect(ValueError, "expected 1", il.Dropout, 0.1, 1, counter=torch.zeros(2, dtype=torch.int64))
    d = il.Dropout(0.1, -1, 2 ** 64 + 5)
    assert d.seed == 2 ** 64 - 1 and d.offset == 5
    d.offset = 2 ** 65 + 7
    assert d.offset == 7


def test_dropout_refuses():
    x = torch.zeros((6, 200), dtype=torch.float16)
    f, d = il.iris_dropout, il.Dropout(0.1, 1)
    expect(ValueError, "out is required", f, None, x, d)
    expect(ValueError, "2-D", f, x, x[0], d)
    expect(TypeError, "x must be one of", f, x.double(), x.double(), d)
    expect(ValueError, "out has shape", f, x[:5], x, d)
    expect(TypeError, "out must be float16", f, x.float(), x, d)
    expect(ValueError, "contiguous along", f, torch.zeros((200, 6), dtype=torch.float16).t(), x, d)
    expect(ValueError, "on a GPU", f, x.clone(), x, d)


def test_block_norm_handle_refuses():
    w = torch.zeros(40)
    n = il.BlockNorm
    expect(ValueError, "kind", n, kind="batch")
    expect(TypeError, "Dropout", n, dropout=0.1)
    expect(ValueError, "need post", n, post_w=w)
    expect(TypeError, "pre_w must be", n, pre_w=w.double())
    expect(ValueError, "vector of 40", n, pre_w=w, pre_b=torch.zeros(41))
    expect(TypeError, "one dtype", n, pre_w=w, pre_b=w.half())
    expect(ValueError, "contiguous", n, pre_w=torch.zeros(80)[::2])
    expect(ValueError, "columns", n, pre_w=w, gate=torch.zeros(2, 41), rows_per_gate=3)
    expect(ValueError, "rows_per_gate is required", n, gate=torch.zeros(2, 40))
    expect(ValueError, "positive", n, gate=torch.zeros(2, 40), rows_per_gate=0)
    expect(ValueError, "contiguous along", n, gate=torch.zeros(40, 2).t(), rows_per_gate=3)


def test_handles_are_not_changed_under_their_pointers():
    """What a handle was made of is read once: set anew it would be passed over in
    silence, or its memory freed while the kernels still read it."""
    d = il.Dropout(0.25, 7)
    norm = il.BlockNorm(post=True, gate=torch.zeros(2, 40), rows_per_gate=3, dropout=d)
    assert (d.p, d.seed, d.counter) == (0.25, 7, None)
    assert (norm.cols, norm.post, norm.rows_per_gate) == (40, True, 3) and norm.gate.shape == (2, 40) and norm.dropout is d
    for handle, names in ((d, ("p", "seed", "counter")), (norm, ("cols", "post", "gate", "rows_per_gate", "dropout"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(handle, name, None)


def test_block_norm_refuses_gates_that_no_rows_use():
    x = torch.zeros((0, 40), dtype=torch.float16)
    norm = il.BlockNorm(gate=torch.zeros(2, 40, dtype=torch.float16), rows_per_gate=3)
    expect(ValueError, "gate has 2 rows, expected 0", il.iris_block_norm, x, norm, y=x, r=x.clone())


def test_block_norm_refuses():
    x, norm = torch.zeros((6, 40), dtype=torch.float16), il.BlockNorm(pre_w=torch.zeros(40, dtype=torch.float16))
    f, b = il.iris_block_norm, il.iris_block_norm_bwd
    expect(TypeError, "BlockNorm", f, x, None, n=x)
    expect(ValueError, "40 columns", f, x[:, :39], norm, n=x[:, :39])
    expect(TypeError, "float16 or bfloat16", f, x, norm, n=x.float())
    expect(TypeError, "or float32", f, x, norm, n=x.bfloat16())          # a stream of fp16 beside bf16
    expect(TypeError, "or float32", f, x.float(), norm, n=x.bfloat16())  # weights of fp16 beside bf16
    gated = il.BlockNorm(gate=torch.zeros((3, 40)), rows_per_gate=3)
    expect(ValueError, "gate has 3 rows, expected 2", f, x, gated, y=x, n=x)
    expect(ValueError, "must be a matrix", f, x, il.BlockNorm(gate=torch.zeros(40), rows_per_gate=3), y=x, n=x)
    expect(ValueError, "on a GPU", f, x, il.BlockNorm(), n=x.clone())
    expect(ValueError, "on a GPU", f, x, norm, n=x.clone())
    expect(ValueError, "stats has shape", f, x, il.BlockNorm(), stats=torch.zeros(6, 3))
    expect(ValueError, "dgate needs", b, x, x, None, il.BlockNorm(), dgate=torch.zeros(40))
    expect(ValueError, "dpre_w has shape", b, None, x, None, il.BlockNorm(), dpre_w=torch.zeros(39))
    expect(TypeError, "dpre_w must be float32", b, None, x, None, il.BlockNorm(), dpre_w=torch.zeros(40, dtype=torch.float16))


def test_mm_act_refuses():
    A, B = empty(6, 200), empty(30, 200, 128)
    C = torch.zeros((6, 30), dtype=torch.float16)
    f, b = il.iris_fp8_mm_act, il.iris_fp8_mm_act_bwd
    expect(TypeError, "Fp8", f, C, A, C)
    expect(ValueError, "expected \\(30, 200\\)", f, C, A, empty(30, 201, 128))
    expect(ValueError, "act must be one of none", f, C, A, B, act="tanh")
    expect(ValueError, "on a GPU", f, C, A, B)
    expect(TypeError, "one of float16", f, C.double(), A, B)
    expect(ValueError, "C is required", b, None, A, B, C, "relu")
    expect(ValueError, "z is required", b, C, A, B, None, "relu")


# ---------------------------------------------------------------- the library

def drop(p=0.1, at=None):
    return _Drop(p, 1, 2, at)


def call_dropout(out=P, x=Q, res=None, t=1, ld=40, alpha=1.0, d=None, rows=6, cols=40, sums=None, ws=None, wsb=0):
    d = drop() if d is None else d
    return _lib.iris_dropout(out, ld, x, ld, res, ld, t, alpha, ctypes.byref(d), sums, rows, cols, ws, wsb, None)


def test_dropout_status_codes():
    assert call_dropout(out=None) == INVALID and call_dropout(x=None) == INVALID
    assert call_dropout(t=4) == INVALID and call_dropout(t=0) == INVALID
    assert call_dropout(x=ODD) == ALIGNMENT
    assert call_dropout(ld=39) == INVALID and call_dropout(ld=1 << 23) == UNSUPPORTED
    assert call_dropout(rows=-1) == INVALID and call_dropout(cols=-1) == INVALID
    assert call_dropout(rows=(1 << 30) + 1) == UNSUPPORTED and call_dropout(cols=(1 << 22) + 1, ld=1 << 22) == UNSUPPORTED
    assert call_dropout(x=P) == INVALID and call_dropout(res=P) == INVALID       # in place
    for p in (-0.1, 1.0, 1.5, float("nan"), 1 - 2.0 ** -18):
        assert call_dropout(d=drop(p)) == INVALID
    assert call_dropout(d=drop(0.1, 0x100004)) == ALIGNMENT
    assert call_dropout(alpha=float("inf")) == INVALID
    assert call_dropout(sums=P) == INVALID and call_dropout(sums=Q) == INVALID and call_dropout(sums=ODD) == ALIGNMENT
    need = il.iris_dropout_workspace_size(6, 40)
    assert need > 0 and call_dropout(sums=R, ws=S, wsb=need - 1) == WORKSPACE and call_dropout(sums=R, ws=S + 8, wsb=need) == ALIGNMENT
    assert il.iris_dropout_workspace_size(-1, 40) == 0 and il.iris_dropout_workspace_size(1 << 30, 1 << 22) <= 32 << 20
    assert call_dropout(rows=0, out=None, x=None) == 0 and call_dropout(cols=0, out=None, x=None) == 0


def test_a_factor_that_leaves_32_bits_is_refused():
    """alpha is finite, alpha / (1 - p) in 32 bits is not: 0 times it would be NaN."""
    top = torch.finfo(torch.float32).max
    assert call_dropout(rows=0, alpha=top, d=drop(0.0)) == 0 and call_dropout(rows=0, alpha=top, d=drop(0.5)) == INVALID
    half = drop(0.5)
    assert call_norm(norm_args(alpha=top, drop=ctypes.pointer(half)), y=R) == INVALID


def norm_args(**kw):
    a = dict(kind=1, type=2, stream_type=2, param_type=2, gate_type=2, post=0, eps=1e-6, w_offset=0.0, alpha=1.0)
    a.update(kw)
    return _Norm(**a)


def call_norm(norm=None, r=None, n=P, q=None, stats=None, x=Q, y=None, rows=6, cols=40, ld=None):
    ld = cols if ld is None else ld
    norm = norm_args() if norm is None else norm
    return _lib.iris_block_norm(r, ld, n, ld, q, stats, x, ld, y, ld, ctypes.byref(norm), rows, cols, None)


def test_block_norm_status_codes():
    assert _lib.iris_block_norm(None, 40, P, 40, None, None, Q, 40, None, 40, None, 6, 40, None) == INVALID
    for bad in (dict(kind=0), dict(kind=3), dict(type=3), dict(stream_type=1), dict(param_type=1), dict(gate_type=1), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(w_offset=float("inf")), dict(alpha=float("nan")), dict(post=1),
                dict(gate=R), dict(post_w=R)):
        assert call_norm(norm_args(**bad)) == INVALID, bad
    assert call_norm(x=None) == INVALID and call_norm(n=None) == INVALID and call_norm(r=R) == INVALID
    assert call_norm(n=Q) == INVALID and call_norm(y=S, r=S) == INVALID
    assert call_norm(norm_args(pre_w=ODD)) == ALIGNMENT and call_norm(stats=0x100008) == ALIGNMENT and call_norm(x=ODD) == ALIGNMENT
    assert call_norm(cols=16385) == UNSUPPORTED and call_norm(ld=39) == INVALID
    assert call_norm(norm_args(gate=R, ld_gate=40, rows_per_gate=0), y=S) == INVALID
    assert call_norm(norm_args(gate=R, ld_gate=39, rows_per_gate=3), y=S) == INVALID
    assert call_norm(norm_args(gate=P, ld_gate=40, rows_per_gate=3), y=S) == INVALID     # the output is the gate
    d = drop(1.0)
    assert call_norm(norm_args(drop=ctypes.pointer(d)), y=S) == INVALID
    q = _Fp8(P, Q, 48, 1, 128)
    assert call_norm(n=None, q=ctypes.byref(q)) == UNSUPPORTED
    assert call_norm(rows=0, n=None, x=None) == 0 and call_norm(cols=0, n=None, x=None, ld=0) == 0


def call_bwd(norm=None, dx=P, dy=None, sums=(None,) * 4, dgate=None, dn=Q, dr=None, r=R, y=None, stats=S, rows=600, cols=40,
             ws=None, wsb=0):
    norm = norm_args() if norm is None else norm
    ld = cols
    return _lib.iris_block_norm_bwd(dx, ld, dy, ld, *sums, dgate, dn, ld, dr, ld, r, ld, y, ld, stats, ctypes.byref(norm), rows, cols,
                                    ws, wsb, None)


def test_block_norm_bwd_status_codes():
    assert call_bwd(dx=None) == INVALID and call_bwd(dn=None) == INVALID and call_bwd(r=None) == INVALID
    assert call_bwd(stats=None) == INVALID and call_bwd(stats=S + 8) == ALIGNMENT
    assert call_bwd(dy=0x500000) == INVALID                                    # needs y
    assert call_bwd(dgate=0x500000, y=0x600000) == INVALID                     # needs a gate
    assert call_bwd(sums=(None, None, 0x500000, None), y=0x600000) == INVALID  # needs post
    assert call_bwd(sums=(0x500002, None, None, None)) == ALIGNMENT
    assert call_bwd(dx=Q) == INVALID and call_bwd(dx=R) == INVALID and call_bwd(sums=(P, None, None, None)) == INVALID
    need = il.iris_block_norm_bwd_workspace_size(600, 40)
    assert need > 0 and call_bwd(ws=0x700000, wsb=need - 1) == WORKSPACE and call_bwd(ws=0x700080, wsb=need) == ALIGNMENT
    assert call_bwd(cols=16385) == UNSUPPORTED
    assert call_bwd(rows=0, dx=None, dn=None, r=None, stats=None) == 0
    assert il.iris_block_norm_bwd_workspace_size(-1, 40) == 0 and il.iris_block_norm_bwd_workspace_size(5, 16385) == 0
    assert max(il.iris_block_norm_bwd_workspace_size(r, c) for r in (1, 300, 1 << 30) for c in (1, 4096, 8192, 16384)) <= 128 << 20


def call_mm(C=P, t=2, A=None, B=None, M=6, N=30, K=200, ws=None, wsb=0, ldc=None, z=None, ld_z=30, q=None, bias=None, act=2,
            alpha=1.0, drop=None, residual=None, ld_residual=30):
    A = _Fp8(0x1000000, 0x2000000, 208, 4, 1) if A is None else A
    B = _Fp8(0x3000000, 0x4000000, 208, 4, 128) if B is None else B
    return _lib.iris_fp8_mm_act(C, t, N if ldc is None else ldc, z, ld_z, q, ctypes.byref(A), ctypes.byref(B), bias, act, alpha, drop,
                                residual, ld_residual, M, N, K, ws, wsb, None)


def test_mm_act_status_codes():
    assert call_mm(C=None) == INVALID and call_mm(t=4) == INVALID and call_mm(act=5) == INVALID and call_mm(act=-1) == INVALID
    assert call_mm(ldc=29) == INVALID and call_mm(C=ODD) == ALIGNMENT and call_mm(bias=ODD) == ALIGNMENT
    assert call_mm(z=Q, ld_z=29) == INVALID and call_mm(residual=Q, ld_residual=29) == INVALID
    assert call_mm(z=P, ld_z=30) == INVALID and call_mm(residual=P, ld_residual=30) == INVALID and call_mm(bias=P) == INVALID
    assert call_mm(alpha=float("nan")) == INVALID
    d = drop(-1.0)
    assert call_mm(drop=ctypes.pointer(d)) == INVALID
    assert call_mm(A=_Fp8(0x1000000, 0x2000000, 208, 4, 128)) == UNSUPPORTED
    assert call_mm(A=_Fp8(0x1000000, 0x2000000, 208, 3, 1)) == ALIGNMENT
    assert call_mm(K=(1 << 21) + 1) == UNSUPPORTED and call_mm(M=-1) == INVALID
    q = _Fp8(P, Q, 32, 1, 1)
    assert call_mm(q=ctypes.pointer(q)) == INVALID            # C and q share memory
    q = _Fp8(Q, R, 32, 1, 128)
    assert call_mm(q=ctypes.pointer(q)) == UNSUPPORTED
    assert call_mm(M=0, C=None) == 0 and call_mm(N=0, C=None, ldc=0) == 0
    need = il.iris_fp8_mm_act_workspace_size(6, 30, 200, torch.bfloat16, to8=True)
    q = _Fp8(Q, R, 32, 1, 1)
    assert need > 0 and call_mm(q=ctypes.pointer(q), ws=0x700000, wsb=need - 1) == WORKSPACE
    assert il.iris_fp8_mm_act_workspace_size(-1, 3, 3) == 0


def test_mm_act_bwd_status_codes():
    A, B = _Fp8(0x1000000, 0x2000000, 208, 4, 1), _Fp8(0x3000000, 0x4000000, 208, 4, 128)

    def call(C=P, dbias=None, z=Q, act=2, M=6, N=30, ws=None, wsb=0, alpha=1.0):
        return _lib.iris_fp8_mm_act_bwd(C, 2, 30, dbias, ctypes.byref(A), ctypes.byref(B), z, 30, act, alpha, None, M, N, 200, ws, wsb,
                                        None)
    assert call(C=None) == INVALID and call(z=None) == INVALID and call(act=0) == INVALID and call(act=9) == INVALID
    assert call(z=P) == INVALID and call(dbias=P) == INVALID and call(dbias=ODD) == ALIGNMENT
    assert call(alpha=float("inf")) == INVALID
    need = il.iris_fp8_mm_act_workspace_size(6, 30, 200, torch.bfloat16, dbias=True)
    assert need > 0 and call(dbias=R, ws=0x700000, wsb=need - 1) == WORKSPACE
    assert call(M=0, C=None, z=None) == 0 and call(N=0, C=None, z=None) == 0
