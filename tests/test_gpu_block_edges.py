"""The block operators where values are not finite."""
import math

import pytest
import torch

import block_ref as bref
import gemm_collective_tile_amd as il
from gpu_util import note
from test_gpu_block import OFFSET, SEED
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
