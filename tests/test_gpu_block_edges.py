"""The block operators where values are not finite, and in the far tails."""
import math

import numpy as np
import pytest
import torch

import block_ref as bref
import gemm_collective_tile_amd as il
from gpu_util import note
from test_gpu_block import OFFSET, SEED, values
from test_gpu_fp8 import DT

INF, NAN = float("inf"), float("nan")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,cols,every", [(1, 8, 1), (40, 300, 7), (700, 1376, 100), (700, 1003, 256), (300, 4096, 300), (130, 4100, 50),
                                             (20, 9000, 3)])
def test_dropped_values_that_are_not_finite_leave_the_gates_gradient_alone(rows, cols, every, dtype):
    """What the mask drops becomes 0, whatever it held: in the forward pass as in the gate's gradient."""
    note(f"gate's gradient {rows}x{cols} {dtype}, NaN and infinities in dropped places")
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    x, y, dn = (torch.randn((rows, cols), device="cuda", generator=g).to(DT[dtype]) for _ in range(3))
    gate = torch.randn((-(-rows // every), cols), device="cuda", generator=g)
    norm = il.BlockNorm(gate=gate, rows_per_gate=every, alpha=0.7, dropout=il.Dropout(0.4, SEED, OFFSET))
    dropped = torch.from_numpy(bref.mask(rows, cols, 0.4, SEED, OFFSET) == 0).cuda()
    bad = torch.where(torch.rand((rows, cols), device="cuda", generator=g) < 0.5, INF, NAN).to(y.dtype)
    results = []
    for wild in (False, True):
        yy = torch.where(dropped, bad if wild else torch.zeros_like(bad), y)
        r, dx, dy = (torch.empty_like(x) for _ in range(3))
        stats, dgate, dw = torch.empty((rows, 4), device="cuda"), torch.empty_like(gate), torch.empty(cols, device="cuda")
        il.iris_block_norm(x, norm, y=yy, r=r, stats=stats)
        il.iris_block_norm_bwd(dx, r, stats, norm, dn=dn, dr=x, y=yy, dy=dy, dgate=dgate, dpre_w=dw)
        results.append((r, stats, dx, dy, dw, dgate))
    for a, b, name in zip(*results, ("r", "stats", "dx", "dy", "dpre_w", "dgate")):
        assert bool(b.isfinite().all()), name
        assert torch.equal(a, b), name
    kept = torch.where(dropped, torch.zeros_like(y), y)   # and what is kept shows
    i, j = (~dropped).nonzero()[-1].tolist()
    kept[i, j] = INF
    il.iris_block_norm_bwd(None, r, stats, norm, dr=x, y=kept, dgate=dgate)
    assert not math.isfinite(float(dgate[i // every, j])) and int((~dgate.isfinite()).sum()) == 1


def slopes(act, z, dtype, M):
    """act'(z) by way of the backward product of ones."""
    n = len(z)
    ones, one = il.iris_fp8_empty(M, 1), il.iris_fp8_empty(n, 1)
    il.iris_fp8_quantize(torch.ones((M, 1), device="cuda"), ones)
    il.iris_fp8_quantize(torch.ones((n, 1), device="cuda"), one)
    C = torch.full((M, n), NAN, dtype=DT[dtype], device="cuda")
    il.iris_fp8_mm_act_bwd(C, ones, one, torch.tensor(z, device="cuda").expand(M, n).to(DT[dtype]).contiguous(), act)
    return C


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M", [3, 90, 200])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_at_infinity(act, M, dtype):
    """1 and 0, the limits: fp16 holds a z of 65520 and more as an infinity."""
    note(f"slope of {act} at infinity, {M} rows, {dtype}")
    C = slopes(act, [INF, -INF, 0.5], dtype, M)
    assert bool((C[:, 0] == 1).all()) and bool((C[:, 1] == 0).all()), (C[0], C[-1])
    assert np.all(np.abs(values(C)[:, 2] - bref.slope(np.array(0.5), act)) <= 2.0 ** -8)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_a_kept_z_beyond_fp16_has_a_gradient(act):
    """The forward pass gives 90000 in 8 bits and keeps z in fp16, as an infinity; the backward pass goes on from it."""
    A, B = il.iris_fp8_empty(200, 1), il.iris_fp8_empty(16, 1)
    il.iris_fp8_quantize(torch.full((200, 1), 300.0, device="cuda"), A)
    il.iris_fp8_quantize(torch.tensor([300.0, -300.0] * 8, device="cuda").reshape(16, 1), B)
    z, q = torch.empty((200, 16), dtype=torch.float16, device="cuda"), il.iris_fp8_empty(200, 16)
    il.iris_fp8_mm_act(None, A, B, act=act, z=z, q=q, dtype=torch.float16)
    assert bool(z[:, ::2].isposinf().all()) and bool(z[:, 1::2].isneginf().all())
    h = q.codes.float() * q.scales.float()
    assert bool(((h[:, ::2] - 288.0 ** 2).abs() <= 2.0 ** -4 * 288.0 ** 2).all()) and bool((h[:, 1::2] == 0).all())
    dh, C = il.iris_fp8_empty(200, 1), torch.full_like(z, NAN)
    il.iris_fp8_quantize(torch.ones((200, 1), device="cuda"), dh)
    one = il.iris_fp8_empty(16, 1)
    il.iris_fp8_quantize(torch.ones((16, 1), device="cuda"), one)
    il.iris_fp8_mm_act_bwd(C, dh, one, z, act)
    assert bool((C[:, ::2] == 1).all()) and bool((C[:, 1::2] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M", [3, 90, 200])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_at_nan(act, M, dtype):
    """The backward pass shows a NaN where the forward pass does."""
    note(f"slope of {act} at NaN, {M} rows, {dtype}")
    C = slopes(act, [1.0, NAN, -1.0, 0.0], dtype, M)
    assert bool(C[:, 1].isnan().all()) and bool(C[:, [0, 2, 3]].isfinite().all())
    if act == "relu":
        assert C[0, [0, 2, 3]].tolist() == [1.0, 0.0, 0.0]


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 200])
def test_gelus_far_tail_keeps_its_digits_in_fp32(M):
    """Relative to its value. The tail's polynomial is within 9.0e-8, its steps and the product with exp add up to
    4.3e-7 with it (in 32 bits with an exact exp and quotient); exp2 and the quotient are good to an ulp, 1.2e-7, the
    latter counted twice for what follows from it; the last product 6e-8: 8.5e-7, so 16 * 2^-24."""
    z = -np.linspace(0.0, 12.8, 4099).astype(np.float32)[1:]
    n = len(z)
    A, B = il.iris_fp8_empty(M, 0), il.iris_fp8_empty(n, 0)
    C = torch.full((M, n), NAN, device="cuda")
    il.iris_fp8_mm_act(C, A, B, act="gelu", bias=torch.from_numpy(z).cuda())
    want = bref.act(z.astype(np.float64), "gelu")
    rel = np.abs(values(C) / want - 1.0).max()
    assert rel <= 16 * 2.0 ** -24, rel
    # the slope, of what it is the difference of: Phi and z phi
    C = slopes("gelu", z.tolist(), "fp32", M)
    zd = z.astype(np.float64)
    phi = np.exp(-0.5 * zd * zd) / math.sqrt(2.0 * math.pi)
    size = bref.act(zd, "gelu") / zd + np.abs(zd) * phi
    rel = (np.abs(values(C) - bref.slope(zd, "gelu")) / size).max()
    assert rel <= 16 * 2.0 ** -24, rel
