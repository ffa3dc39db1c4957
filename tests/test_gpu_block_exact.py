"""Products with an epilogue on the GPU, to the bit: codes -1, 0 and 1 under scales 1 and 2,
whole numbers beside them and a dropout of one half, whose factor is 2. All sums stay
below 256, which bf16 holds, so every output has one right value in every type and any
order of the sums, on each tile, whole and ragged, and each way to split and join. A row
that is missing, read twice or taken from another strip shows, in the bias's
gradient too: its sums stay below 2^24, and C's type rounds them once.

The activations that are not exact follow in the largest tile, with the bounds of
test_gpu_block.
"""
import functools

import numpy as np
import pytest
import torch

import block_ref as bref
import fp8_ref as ref
import gemm_collective_tile_amd as il
from fp8_plan import ACT_OF_EACH_PLAN, plan_act
from gpu_util import note
from test_gpu_block import OFFSET, SEED, check_mm_act, check_mm_act_bwd, out_of
from test_gpu_fp8 import DT, assert_untouched, fresh, parts, put

ONE, MINUS = 0x38, 0xB8   # e4m3 codes of 1 and -1


@functools.lru_cache(maxsize=2)
def operands(M, N, K, block):
    """A (M, K), B (N, K) and their product in 64 bits, on the GPU."""
    rng = np.random.default_rng(M + N + K)
    keep = 0.2 * (1105 / K) ** 0.5   # sums of K terms of about the same size for all K
    made = []
    for rows, b in ((M, 1), (N, block)):
        codes = np.where(rng.random((rows, K)) < keep, np.where(rng.random((rows, K)) < 0.5, ONE, MINUS), 0).astype(np.uint8)
        scales = rng.integers(127, 129, size=(-(-rows // b), -(-K // ref.BLK))).astype(np.uint8)
        made.append((put(codes, scales, b), torch.from_numpy(ref.values(codes, scales, b)).cuda()))
    (A, a), (B, b) = made
    return A, B, a @ b.t().contiguous()


@functools.lru_cache(maxsize=1)
def mask(M, N):
    return torch.from_numpy(bref.mask(M, N, 0.5, SEED, OFFSET)).cuda()


def whole_numbers(M, N, most, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, (M, N), device="cuda", generator=g).double()


def placed(x, dtype, pitch, offset):
    """x at a row pitch and an offset, NaN around it."""
    store = torch.full((offset + x.shape[0] * pitch + 8,), float("nan"), dtype=DT[dtype], device="cuda")
    t = torch.as_strided(store, x.shape, (pitch, 1), offset)
    t.copy_(x)
    return t


def same(t, want, what):
    want = want.to(t.dtype)
    if not torch.equal(t, want):
        bad = ~(t == want)
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {at}: {float(t[tuple(at)])}, "
                             f"not {float(want[tuple(at)])}")


def layout(N):
    """Pitches and an offset of C, z and the residual, all different: aligned ones where N is whole."""
    return ((N + 8, N + 16, N), 8) if N % 8 == 0 else ((N + 3, N, N + 6), 3)


# activation, bias, z, residual, dropout, outputs
WAYS = [("none", True, False, True, True, "C"), ("relu", True, True, False, False, "q"), ("relu", True, True, True, True, "Cq"),
        ("relu", False, True, True, False, "C"), ("none", False, False, False, False, "C")]


@pytest.mark.gpu
@pytest.mark.parametrize("way", range(len(WAYS)))
@pytest.mark.parametrize("dtype,M,N,K,want", ACT_OF_EACH_PLAN)
def test_mm_act_to_the_bit(dtype, M, N, K, want, way):
    act, with_bias, with_z, with_res, dropped, outs = WAYS[way]
    if "q" not in outs:
        assert plan_act(M, N, K, dtype) == want
    elif want[1] >= 128:
        assert plan_act(M, N, K, dtype, to8=True) == want
    note(f"exact mm act {M}x{N}x{K} {dtype} {want} {WAYS[way]}")
    A, B, v = operands(M, N, K, 128 if way % 2 else 1)
    (pc, pz, pr), offset = layout(N)
    bias = whole_numbers(1, N, 3, 1)[0] if with_bias else None
    res = whole_numbers(M, N, 15, 2) if with_res else None
    v = v if bias is None else v + bias
    c = v.clamp(min=0.0) if act == "relu" else v
    c = c * mask(M, N) if dropped else c
    c = c if res is None else c + res
    assert float(c.abs().max()) <= 256 and float(v.abs().max()) <= 256, "the case is not exact in bf16"
    C, c_in = out_of(M, N, dtype, pc, offset) if "C" in outs else (None, None)
    z, z_in = out_of(M, N, dtype, pz, offset) if with_z else (None, None)
    q = fresh(M, N) if "q" in outs else None
    il.iris_fp8_mm_act(C, A, B, act=act, bias=None if bias is None else bias.to(DT[dtype]), z=z, q=q, dtype=DT[dtype],
                       residual=None if res is None else placed(res, dtype, pr, offset),
                       dropout=il.Dropout(0.5, SEED, OFFSET) if dropped else None)
    if C is not None:
        same(C, c, "C")
        assert c_in()
    if z is not None:
        same(z, v, "z")
        assert z_in()
    if q is not None:
        q2 = il.iris_fp8_empty(M, N)
        il.iris_fp8_quantize(c.float(), q2)
        assert all(np.array_equal(a, b) for a, b in zip(parts(q), parts(q2))), "8-bit output"
        assert_untouched(q, "8-bit output")


@pytest.mark.gpu
@pytest.mark.parametrize("dropped,with_dbias", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("dtype,M,N,K,want", ACT_OF_EACH_PLAN)
def test_mm_act_bwd_to_the_bit(dtype, M, N, K, want, dropped, with_dbias):
    assert plan_act(M, N, K, dtype) == want
    note(f"exact mm act backward {M}x{N}x{K} {dtype} {want} dropout {dropped} dbias {with_dbias}")
    A, B, v = operands(M, N, K, 128 if dropped else 1)
    (pc, pz, _), offset = layout(N)
    z = whole_numbers(M, N, 4, 3)
    c = torch.where(z > 0, v, torch.zeros_like(v))   # relu's slope is 0 at 0
    c = c * mask(M, N) if dropped else c
    assert float(c.abs().max()) <= 256 and float(c.abs().sum(0).max()) < 2 ** 24, "the case is not exact"
    C, c_in = out_of(M, N, dtype, pc, offset)
    dbias = torch.full((N,), float("nan"), dtype=DT[dtype], device="cuda") if with_dbias else None
    il.iris_fp8_mm_act_bwd(C, A, B, placed(z, dtype, pz, offset), "relu", dbias=dbias,
                           dropout=il.Dropout(0.5, SEED, OFFSET) if dropped else None)
    same(C, c, "C")
    assert c_in()
    if with_dbias:
        same(dbias, c.sum(0), "dbias")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,N", [("fp16", 4104), ("bf16", 4103), ("bf16", 4104), ("fp32", 5000), ("fp32", 5003)])
def test_curved_activations_in_the_largest_tile(dtype, N):
    M, K = 3005, 1105
    assert plan_act(M, N, K, dtype) == plan_act(M, N, K, dtype, to8=True) == (256, 256, 1)
    check_mm_act(M, N, K, dtype, 128, "gelu_tanh", 0.2, True, False, True, "Cq")
    check_mm_act(M, N, K, dtype, 128, "silu", 0.0, False, True, False, "C")
    check_mm_act_bwd(M, N, K, dtype, 128, "gelu_tanh", 0.2, True)
