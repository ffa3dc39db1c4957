"""The norm around a block behind the fp16 products with collectives: a row-parallel
projection's summed output is added to the residual stream and normed for the next block."""
import pytest
import torch

import block_ref as bref
import gemm_collective_tile_amd as il
import oracle
import workloads as wl
from gpu_util import assert_close, empty, host, note
from test_gpu_block import OFFSET, SEED, close, close8, out_of, values
from test_gpu_fp8 import fresh


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,W", [(200, 320, 72, 3), (257, 1376, 344, 2)])
def test_norm_after_matmul_all_reduce(M, N, K, W):
    note(f"matmul_all_reduce {M}x{N}x{K} W {W}, then block norm")
    w = wl.Workload("case", "mm_ar", M=M, N=N, K=K, W=W, a_std=1.0, b_std=K ** -0.5)
    inp = wl.make_inputs(w, seed=10)
    C, y = empty((M, N)), empty((M, N))
    il.iris_mm_ar_local(y, C, inp["A"].cuda(), inp["B"].cuda(), [p.cuda() for p in inp["partials"]], W, bias=inp["bias"].cuda())
    x = torch.randn((M, N), generator=torch.Generator().manual_seed(1)).cuda()
    gate, pre_w = torch.linspace(-1, 1, N, device="cuda"), torch.linspace(0.5, 1.5, N, device="cuda")
    norm = il.BlockNorm(eps=1e-5, pre_w=pre_w, post=True, gate=gate, alpha=0.7, dropout=il.Dropout(0.1, SEED, OFFSET))
    r, r_in = out_of(M, N, "fp32")
    n, n_in = out_of(M, N, "fp16")
    q, stats = fresh(M, N), torch.empty((M, 4), device="cuda")
    il.iris_block_norm(x, norm, y=y, r=r, n=n, q=q, stats=stats)   # behind the product on its stream, without a wait
    assert_close(y, oracle.matmul_all_reduce(host(inp["A"]), host(inp["B"]), [host(p) for p in inp["partials"]], W,
                                             bias=host(inp["bias"])), "y")
    want, off = bref.block_norm(values(x), values(y), eps=1e-5, pre_w=values(pre_w), post=True, gate=values(gate)[None, :], alpha=0.7,
                                m=bref.mask(M, N, 0.1, SEED, OFFSET))
    close(r, want["r"], off["r"], "fp32", "r")
    close(n, want["n"], off["n"], "fp16", "n")
    close8(q, want["n"], off["n"], "q")
    close(stats, want["stats"], off["stats"], "fp32", "stats")
    assert r_in() and n_in()
