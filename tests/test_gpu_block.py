"""The block operators on the GPU (dropout, the norms around a block, the 8-bit product
with an epilogue) against the plain 64-bit forms of block_ref.

Bounds. block_ref gives, beside each value, what 32-bit sums and products may be off
(magnitudes times 2^-24 times the roundings on the way); then one rounding to the
output's type: half a step, and half of fp16's subnormal step 2^-24. Products: the sum is
within (K + 2) 2^-23 sum |a b| of the exact one, in 16-bit types also 2^-10 sum |a b|
(what the matrix unit drops). An activation passes an error on with its slope, at most
1.13 (gelu, at sqrt 2) for all of them, and adds 1e-5 of its own value: the exponent's
product rounds to |u| / 2 ulps, and |u| < 128 where exp(u) is not 0 or infinite: 64 * 2^-24
* 2, and 4.2e-7 of gelu's fitted tail. A slope is off by at most 1.3e-5 (its terms, each at
most 1.2, have 1e-5). 8-bit outputs: half an e4m3 step more, at either neighbouring scale
where the block's largest magnitude is within its bound of a border.
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

import block_ref as bref
import fp8_ref as ref
import gemm_collective_tile_amd as il
from gpu_util import note
from test_gpu_fp8 import DT, ULP, assert_untouched, fresh, from_gpu, on_gpu, parts, sample

_plan = il._lib["_ZN4iris16fp8_mm_plan_wideElllbi"]


class Plan(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("splits", ctypes.c_int32), ("split_steps", ctypes.c_int32),
                ("ws_bytes", ctypes.c_size_t)]


_plan.restype, _plan.argtypes = Plan, [ctypes.c_int64] * 3 + [ctypes.c_bool, ctypes.c_int32]


def plan(M, N, K, dtype, to8=False):
    p = _plan(M, N, K, dtype == "fp32", 128 if to8 else 0)
    return (p.bm, p.bn, p.splits) if p.bm else (0, 0, 1)


def values(t):
    return t.detach().double().cpu().numpy()


def close(t, want, off, dtype, what):
    """t (rounded to dtype) against `want`, which 32-bit arithmetic may miss by `off`."""
    got = values(t)
    bound = off + ULP[dtype] * (np.abs(want) + off) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    ok = np.abs(got - want) <= bound
    if dtype == "fp16":   # 65520, half a step over the largest value, and what is beyond round to infinity
        ok |= (got == np.copysign(np.inf, want)) & (np.abs(want) + off >= 65520.0)
    bad = ~ok
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][0], want[bad][0], (off + 0 * want)[bad][0])


def close8(q, want, off, what):
    """An 8-bit output against `want`, itself off by `off` before its rounding."""
    codes, scales = parts(q)
    off = off + np.zeros_like(want)
    least, most = (ref.block_amax(np.maximum(np.abs(want) + s * off, 0.0), 1) for s in (-1, 1))
    lo, hi = np.where(least == 0, 1, ref.scale_bytes(least)), ref.scale_bytes(most)
    # a block that may be all zeros may have the scale of one: 1, byte 127
    assert np.all((scales >= lo) & (scales <= hi) | (least == 0) & (scales == 127)), f"{what}: scales"
    sc = ref.spread(scales, 1, codes.shape)
    got = ref.decode(codes) * sc
    a = np.abs(want) + off
    step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(a / sc, 2.0 ** -30))) - 3), ref.SUB)
    bad = ~(np.abs(got - want) <= 0.5 * step * sc + off)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][0], want[bad][0])
    assert_untouched(q, what)


def out_of(rows, cols, dtype, pitch=None, offset=0):
    """An output full of NaN inside memory full of NaN, and a check that its padding stays so."""
    pitch = cols if pitch is None else pitch
    store = torch.full((offset + rows * pitch + 8,), float("nan"), dtype=DT[dtype], device="cuda")
    t = torch.as_strided(store, (rows, cols), (pitch, 1), offset)

    def untouched():
        rest = store.clone()
        torch.as_strided(rest, (rows, cols), (pitch, 1), offset).fill_(float("nan"))
        return bool(rest.isnan().all())
    return t, untouched


SEED, OFFSET = 0x0123456789ABCDEF, 0xFEDCBA9876543210

# ----------------------------------------------------------------- dropout


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols,pitch,offset", [(1, 1, None, 0), (1, 4096, None, 0), (3, 7, 9, 1), (5, 129, None, 0),
                                                    (37, 1376, 1376, 0), (200, 333, 340, 3), (64, 256, 264, 8), (9, 8, 8, 0),
                                                    (1000, 15, 15, 0)])
def test_dropout(rows, cols, pitch, offset, dtype):
    note(f"dropout {rows}x{cols} {dtype} pitch {pitch} offset {offset}")
    x, xv = on_gpu(sample(rows, cols, rows + cols), dtype, pitch, offset)
    res, rv = on_gpu(sample(rows, cols, rows + cols + 1), dtype, None if pitch is None else pitch + 8, offset)
    for p, residual, alpha in ((0.1, True, 0.7), (0.6, False, 1.0), (0.0, True, -2.0), (1e-6, False, 1.0), (0.99999, False, 1.0)):
        out, untouched = out_of(rows, cols, dtype, pitch, offset)
        il.iris_dropout(out, x, il.Dropout(p, SEED, OFFSET), residual=res if residual else None, alpha=alpha)
        m = bref.mask(rows, cols, p, SEED, OFFSET)
        want, size = alpha * m * xv, np.abs(alpha * m * xv)
        if residual:
            want, size = want + rv, size + np.abs(rv)
        close(out, want, 3 * bref.EPS32 * size, dtype, (p, residual))
        if not residual:
            assert np.array_equal(values(out) == 0, (m == 0) | (xv == 0)) or dtype == "fp16"
        assert untouched()
    out, _ = out_of(rows, cols, dtype)
    il.iris_dropout(out, x, None, alpha=1.0)
    assert np.array_equal(values(out), xv)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols,pitch,offset", [(1, 1, None, 0), (1, 4096, None, 0), (5, 129, 131, 1), (16, 128, None, 0),
                                                    (37, 1376, None, 0), (200, 333, 340, 3), (5000, 40, None, 0), (2000, 264, 272, 8)])
def test_dropout_sums(rows, cols, pitch, offset, dtype):
    note(f"dropout with sums {rows}x{cols} {dtype} pitch {pitch} offset {offset}")
    x, xv = on_gpu(sample(rows, cols, rows + cols), dtype, pitch, offset)
    res, rv = on_gpu(sample(rows, cols, rows + cols + 1), dtype, pitch, offset)
    for p, residual, alpha in ((0.1, True, 0.7), (0.0, False, 1.0), (0.6, False, 0.5)):
        m = bref.mask(rows, cols, p, SEED, OFFSET)
        want, size = alpha * m * xv, np.abs(alpha * m * xv)
        if residual:
            want, size = want + rv, size + np.abs(rv)
        two = []
        for _ in range(2):
            out, untouched = out_of(rows, cols, dtype, pitch, offset)
            sums = torch.full((cols,), float("nan"), dtype=DT[dtype], device="cuda")
            il.iris_dropout(out, x, il.Dropout(p, SEED, OFFSET), residual=res if residual else None, alpha=alpha, sums=sums)
            two.append(sums)
            assert untouched()
        close(out, want, 3 * bref.EPS32 * size, dtype, (p, residual))
        close(sums, want.sum(0), ((rows + 32) * bref.EPS32 * size).sum(0), dtype, "sums")
        assert torch.equal(*two)
    ws = torch.full((il.iris_dropout_workspace_size(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    il.iris_dropout(out, x, il.Dropout(p, SEED, OFFSET), alpha=alpha, sums=two[0], workspace=ws)
    assert torch.equal(*two)
    none = torch.empty((0, cols), dtype=DT[dtype], device="cuda")
    il.iris_dropout(torch.empty_like(none), none, None, sums=sums)
    assert bool((sums == 0).all())


@pytest.mark.gpu
def test_dropout_drops_what_is_not_finite_and_keeps_the_rest_so():
    x = torch.full((64, 256), float("inf"), dtype=torch.bfloat16, device="cuda")
    x[::2] = float("nan")
    out = torch.zeros_like(x)
    il.iris_dropout(out, x, il.Dropout(0.5, 9))
    m = bref.mask(64, 256, 0.5, 9, 0)
    got = values(out)
    assert np.array_equal(got == 0, m == 0)
    assert np.isnan(got[::2][m[::2] > 0]).all() and np.isposinf(got[1::2][m[1::2] > 0]).all()


@pytest.mark.gpu
def test_dropout_of_more_rows_than_a_launch_holds():
    """2^31 pieces of 8 columns and more go in several launches: the mask's rows go on."""
    rows, cols, part = (1 << 22) + 5, 4096, 1 << 22
    note("dropout of 2^34 values")
    x = torch.ones((rows, cols), dtype=torch.float16, device="cuda")
    y = torch.empty((rows, cols), dtype=torch.float16, device="cuda")
    il.iris_dropout(y, x, il.Dropout(0.25, 5, 6))
    for r in (0, part - 1, part, rows - 1):
        close(y[r:r + 1], bref.mask(1, cols, 0.25, 5, 6, row0=r), 0.0, "fp16", r)


@pytest.mark.gpu
def test_dropout_counter_in_a_replayed_graph():
    """A graph that adds to the counter takes a new mask with every replay, the one that the eager call takes too."""
    x, xv = on_gpu(sample(33, 500, 1), "fp32")
    out = torch.zeros((33, 500), device="cuda")
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    d = il.Dropout(0.3, SEED, OFFSET, counter)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        counter.add_(1)
        il.iris_dropout(out, x, d)
    for k in range(1, 5):
        g.replay()
        torch.cuda.synchronize()
        assert int(counter) == k
        m = bref.mask(33, 500, 0.3, SEED, (OFFSET + k) % 2 ** 64)
        close(out, m * xv, 3 * bref.EPS32 * np.abs(m * xv), "fp32", k)
        eager = torch.empty_like(out)
        il.iris_dropout(eager, x, d)
        assert torch.equal(eager, out)
    d.offset = 2 ** 64 - 4    # the sum wraps
    il.iris_dropout(out, x, d)
    m = bref.mask(33, 500, 0.3, SEED, 0)
    close(out, m * xv, 3 * bref.EPS32 * np.abs(m * xv), "fp32", "wrapped")


# ------------------------------------------------------------------- norms

NORM_SHAPES = [(1, 1), (1, 8), (1, 4096), (3, 130), (5, 512), (9, 513), (2, 1000), (7, 1025), (33, 1376), (4, 2049), (3, 4093),
               (2, 5000), (3, 8200), (2, 16384), (2, 16381), (300, 264), (1030, 40)]
# kind, y, post, gate rows (0: none, -1: a vector), p, biases, parameters in fp32, w_offset, stream in fp32
NORM_WAYS = [("rms", True, True, -1, 0.1, False, False, 0.0, True), ("layer", True, True, 2, 0.0, True, False, 0.0, False),
             ("rms", False, False, 0, 0.0, False, True, 1.0, False), ("layer", True, False, 3, 0.25, True, True, 0.0, True),
             ("rms", True, False, 0, 0.0, False, False, 0.0, False), ("layer", False, False, 0, 0.0, True, False, 0.5, True)]


def norm_case(rows, cols, way, dtype, seed, pitch=None, offset=0):
    """(tensors, values, keyword arguments of the plain form, BlockNorm, gate row of every row)."""
    kind, has_y, post, gate, p, biases, p32, w_off, s32 = way
    stream, param = "fp32" if s32 else dtype, "fp32" if p32 else dtype
    rng = np.random.default_rng(seed)
    t, v = {}, {}
    t["x"], v["x"] = on_gpu(sample(rows, cols, seed), stream, pitch, offset)
    if has_y:
        t["y"], v["y"] = on_gpu(sample(rows, cols, seed + 1), dtype, pitch, offset)
    for side in ["pre"] + (["post"] if post else []):
        w, v[side + "_w"] = on_gpu(1.0 - w_off + 0.2 * rng.normal(size=(1, cols)), param, None, offset)
        t[side + "_w"] = w.reshape(-1)
        if biases:
            b, v[side + "_b"] = on_gpu(0.3 * rng.normal(size=(1, cols)), param)
            t[side + "_b"] = b.reshape(-1)
    every, group, g_wide = None, np.zeros(rows, np.int64), None
    if gate:
        every = rows if gate < 0 else min(gate, rows) if rows < 100 else 37
        group = np.arange(rows) // every
        t["gate"], v["gate"] = on_gpu(0.7 * rng.normal(size=(int(group[-1]) + 1, cols)), dtype)
        g_wide = v["gate"][group]
        if gate < 0:
            t["gate"] = t["gate"][0]
    alpha = 0.8 if has_y else 1.0
    drop = il.Dropout(p, SEED + seed, OFFSET) if p > 0 else None
    norm = il.BlockNorm(kind=kind, eps=1e-5, post=post, alpha=alpha, dropout=drop, w_offset=w_off,
                        rows_per_gate=every if gate > 0 else None,
                        **{k: t[k] for k in ("pre_w", "pre_b", "post_w", "post_b", "gate") if k in t})
    plain = {k: v[k].reshape(-1) for k in ("pre_b", "post_b") if k in v}
    plain |= {k: v[k].reshape(-1) + w_off for k in ("pre_w", "post_w") if k in v}
    plain |= {"layer": kind == "layer", "post": post, "gate": g_wide, "alpha": alpha,
              "m": bref.mask(rows, cols, p, SEED + seed, OFFSET) if p > 0 else 1.0}
    return t, v, plain, norm, group, stream


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("way", range(len(NORM_WAYS)))
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_block_norm(rows, cols, way, dtype):
    w = NORM_WAYS[way]
    note(f"block norm {rows}x{cols} {dtype} {w}")
    t, v, plain, norm, _, stream = norm_case(rows, cols, w, dtype, 7 * rows + cols)
    has_y = "y" in t
    want, off = bref.block_norm(v["x"], v.get("y"), eps=1e-5, **plain)
    r, r_in = out_of(rows, cols, stream)
    n, n_in = out_of(rows, cols, dtype)
    q = fresh(rows, cols)
    stats = torch.full((rows, 4), float("nan"), device="cuda")
    il.iris_block_norm(t["x"], norm, y=t.get("y"), r=r if has_y else None, n=n, q=q, stats=stats)
    if has_y:
        close(r, want["r"], off["r"], stream, "r")
    close(n, want["n"], off["n"], dtype, "n")
    close8(q, want["n"], off["n"], "q")
    close(stats, want["stats"], off["stats"], "fp32", "stats")
    assert r_in() and n_in()
    # each output alone has the same bits
    n2, q2, s2 = torch.empty_like(n), fresh(rows, cols), torch.empty_like(stats)
    il.iris_block_norm(t["x"], norm, y=t.get("y"), n=n2)
    il.iris_block_norm(t["x"], norm, y=t.get("y"), q=q2)
    il.iris_block_norm(t["x"], norm, y=t.get("y"), stats=s2)
    assert torch.equal(n, n2) and torch.equal(stats, s2)
    assert all(np.array_equal(a, b) for a, b in zip(parts(q), parts(q2)))


@pytest.mark.gpu
@pytest.mark.parametrize("pitch,offset", [(320, 0), (304, 8), (301, 0), (300, 1), (303, 5)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_block_norm_pitch_and_offset(pitch, offset, dtype):
    note(f"block norm 40x300 {dtype} pitch {pitch} offset {offset}")
    t, v, plain, norm, group, stream = norm_case(40, 300, NORM_WAYS[1], dtype, pitch, pitch, offset)
    want, off = bref.block_norm(v["x"], v["y"], eps=1e-5, **plain)
    r, r_in = out_of(40, 300, stream, pitch, offset)
    n, n_in = out_of(40, 300, dtype, pitch, offset)
    stats = torch.empty((40, 4), device="cuda")
    il.iris_block_norm(t["x"], norm, y=t["y"], r=r, n=n, stats=stats)
    close(r, want["r"], off["r"], stream, "r")
    close(n, want["n"], off["n"], dtype, "n")
    assert r_in() and n_in()
    run_bwd(t, v, plain, norm, group, stream, dtype, 40, 300, pitch, offset)


def run_bwd(t, v, plain, norm, group, stream, dtype, rows, cols, pitch=None, offset=0, with_dn=True, with_dr=True):
    has_y, post, gate = "y" in t, plain["post"], plain["gate"] is not None
    # a stream and its statistics, as a forward pass leaves them
    r, rv = t["x"], v["x"]
    stats = np.zeros((rows, 4))
    stats[:, 2:] = np.concatenate(bref.statistics(rv, plain["layer"], 1e-5)[:2], 1)
    if post:
        stats[:, :2] = np.concatenate(bref.statistics(v["y"], plain["layer"], 1e-5)[:2], 1)
    st = torch.from_numpy(stats).float().cuda()
    stats = st.double().cpu().numpy()
    dn, dnv = on_gpu(sample(rows, cols, cols + 3) / 16, dtype, pitch, offset) if with_dn else (None, None)
    dr, drv = on_gpu(sample(rows, cols, cols + 4) / 16, stream, pitch, offset) if with_dr else (None, None)
    kw = {k: plain[k] for k in ("layer", "post", "gate", "alpha", "m", "pre_w", "post_w", "post_b") if k in plain}
    want, off = bref.block_norm_bwd(rv, stats, dnv, drv, v.get("y"), group=group, **kw)
    outs = {"dx": out_of(rows, cols, stream, pitch, offset)}
    if has_y:
        outs["dy"] = out_of(rows, cols, dtype, pitch, offset)
    sums = [k for k in ("dpre_w", "dpre_b", "dpost_w", "dpost_b", "dgate") if k in want]
    tensors = [{k: torch.full(want[k].shape, float("nan"), device="cuda") for k in sums} for _ in range(2)]
    for got in tensors:
        if gate and norm.gate.dim() == 1:
            got["dgate"] = got["dgate"][0]
        il.iris_block_norm_bwd(outs["dx"][0], r, st, norm, dn=dn, dr=dr, y=t.get("y"), dy=outs["dy"][0] if has_y else None, **got)
    close(outs["dx"][0], want["dx"], off["dx"], stream, "dx")
    if has_y:
        close(outs["dy"][0], want["dy"], off["dy"], dtype, "dy")
    for k in sums:
        close(tensors[0][k].reshape(want[k].shape), want[k], off[k], "fp32", k)
        assert torch.equal(tensors[0][k], tensors[1][k]), k
    assert all(u() for _, u in outs.values())
    # a gradient alone has the same bits
    for k in sums:
        one = torch.full_like(tensors[0][k], float("nan"))
        il.iris_block_norm_bwd(None, r, st, norm, dn=dn, dr=dr, y=t.get("y"), **{k: one})
        assert torch.equal(one, tensors[0][k]), k
    return tensors[0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("way", range(len(NORM_WAYS)))
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_block_norm_bwd(rows, cols, way, dtype):
    note(f"block norm backward {rows}x{cols} {dtype} {NORM_WAYS[way]}")
    case = norm_case(rows, cols, NORM_WAYS[way], dtype, 7 * rows + cols)
    t, v, plain, norm, group, stream = case
    run_bwd(t, v, plain, norm, group, stream, dtype, rows, cols, with_dn=way != 3, with_dr=way != 4)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,every", [(700, 1), (700, 2), (700, 3), (700, 100), (700, 256), (700, 699), (2, 1), (1, 1),
                                        (257, 2), (5000, 1700), (5000, 21)])
def test_block_norm_gates_of_every_length(rows, every):
    """Gates whose rows lie in one workgroup, in several, and begin or end inside one."""
    cols = 2056
    note(f"gates of {every} of {rows} rows")
    t, v, plain, _, _, stream = norm_case(rows, cols, NORM_WAYS[0], "bf16", rows)
    group = np.arange(rows) // every
    gate, gv = on_gpu(np.random.default_rng(every).normal(size=(int(group[-1]) + 1, cols)), "fp32")
    norm = il.BlockNorm(eps=1e-5, post=True, alpha=0.8, dropout=il.Dropout(0.1, SEED + rows, OFFSET), pre_w=t["pre_w"].float(),
                        post_w=t["post_w"].float(), gate=gate, rows_per_gate=every)
    plain["gate"] = gv[group]
    plain["m"] = bref.mask(rows, cols, 0.1, SEED + rows, OFFSET)
    run_bwd(t, v, plain, norm, group, stream, "bf16", rows, cols)


@pytest.mark.gpu
def test_block_norm_of_more_rows_than_a_launch_holds():
    """2^20 rows and more go in several launches: the mask's and the gate's rows go on. The backward pass takes them at once."""
    rows, cols, every, part = (1 << 20) + 77, 24, 1000, 1 << 20
    note("block norm of 2^20 rows")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, y = (torch.randn((rows, cols), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    gate = torch.randn((-(-rows // every), cols), device="cuda", generator=g)
    norm = il.BlockNorm(gate=gate, rows_per_gate=every, dropout=il.Dropout(0.2, 5, 6))
    r, n, stats, q = torch.empty_like(x), torch.empty_like(x), torch.empty((rows, 4), device="cuda"), il.iris_fp8_empty(rows, cols)
    il.iris_block_norm(x, norm, y=y, r=r, n=n, q=q, stats=stats)
    dx, dy, dgate, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gate), torch.empty(cols, device="cuda")
    il.iris_block_norm_bwd(dx, r, stats, norm, dn=n, y=y, dy=dy, dgate=dgate, dpre_w=dw)
    for at in (0, 512 * 1024, part - 40, rows - 80):
        some = slice(at, at + 80)
        m = bref.mask(80, cols, 0.2, 5, 6, row0=at)
        wide = values(gate)[np.arange(at, at + 80) // every]
        want, off = bref.block_norm(values(x[some]), values(y[some]), gate=wide, m=m)
        close(r[some], want["r"], off["r"], "bf16", "r")
        close(n[some], want["n"], off["n"], "bf16", "n")
        close(stats[some], want["stats"], off["stats"], "fp32", "stats")
        part8 = il.Fp8(q.codes[some], q.scales[some])
        got = ref.values(*parts(part8))
        assert np.all(np.abs(got - want["n"]) <= 2.0 ** -4 * np.abs(want["n"]) + 2.0 ** -10 * np.abs(want["n"]).max() + off["n"])
        back, boff = bref.block_norm_bwd(values(r[some]), values(stats[some]), values(n[some]), None, values(y[some]), gate=wide, m=m,
                                         group=np.arange(80))
        close(dx[some], back["dx"], boff["dx"], "bf16", "dx")
        close(dy[some], back["dy"], boff["dy"], "bf16", "dy")
    # gates of the first rows, of rows that two workgroups share, and the last, shorter one
    t = values(dx)
    for k in (0, 1, 2, 3, 500, gate.shape[0] - 1):
        rows_k = slice(k * every, min((k + 1) * every, rows))
        m = bref.mask(rows_k.stop - rows_k.start, cols, 0.2, 5, 6, row0=rows_k.start)
        each = m * t[rows_k] * values(y[rows_k])
        # dx was rounded to bf16, half a step of each term
        bound = (np.abs(each) * (2.0 ** -8 + 1200 * bref.EPS32)).sum(0)
        assert np.all(np.abs(values(dgate[k]) - each.sum(0)) <= bound), k
    hat = (values(r) - values(stats)[:, 2:3]) * values(stats)[:, 3:]
    each = values(n) * hat
    assert np.all(np.abs(values(dw) - each.sum(0)) <= np.abs(each).sum(0) * (2048 + 600) * bref.EPS32)


@pytest.mark.gpu
def test_column_sums_in_graphs_side_by_side_in_workspaces_of_their_own():
    """Two graphs that replay at the same time on two streams, each with its own workspace."""
    graphs, wanted = [], []
    for k in range(2):
        t, v, plain, norm, group, stream = norm_case(900, 2048, NORM_WAYS[0], "bf16", 40 + k)
        stats = torch.ones((900, 4), device="cuda")
        dw, dg = torch.empty(2048, device="cuda"), torch.empty(2048, device="cuda")
        ws = torch.empty(il.iris_block_norm_bwd_workspace_size(900, 2048), dtype=torch.uint8, device="cuda")
        out, sums = torch.empty_like(t["y"]), torch.empty(2048, dtype=torch.bfloat16, device="cuda")
        ws2 = torch.empty(il.iris_dropout_workspace_size(900, 2048), dtype=torch.uint8, device="cuda")

        def run(t=t, norm=norm, stats=stats, dw=dw, dg=dg, ws=ws, out=out, sums=sums, ws2=ws2):
            il.iris_block_norm_bwd(None, t["x"], stats, norm, dn=t["y"], y=t["y"], dpre_w=dw, dgate=dg, workspace=ws)
            il.iris_dropout(out, t["y"], norm.dropout, sums=sums, workspace=ws2)
        run()
        torch.cuda.synchronize()
        wanted.append([x.clone() for x in (dw, dg, sums)])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(10):
                run()
        graphs.append((g, s, (dw, dg, sums), run))   # run holds what the graph reads
    for _ in range(4):
        for _, _, outs, _ in graphs:
            for x in outs:
                x.zero_()
        torch.cuda.synchronize()
        for g, s, _, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, outs, _), want in zip(graphs, wanted):
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.gpu
def test_block_norm_of_zeros_and_of_what_is_not_finite():
    """A row of zeros has a finite norm (eps); NaN and infinities stay in their row."""
    x = torch.randn((9, 600), device="cuda").to(torch.float16)
    x[1] = 0
    clean = torch.empty_like(x)
    norm = il.BlockNorm(kind="layer")
    il.iris_block_norm(x, norm, n=clean)
    assert bool((clean[1] == 0).all()) and bool(clean.isfinite().all())
    x[3, 17], x[5, 599] = float("nan"), float("inf")
    n, q = torch.empty_like(x), fresh(9, 600)
    il.iris_block_norm(x, norm, n=n, q=q)
    keep = [0, 1, 2, 4, 6, 7, 8]
    assert torch.equal(n[keep], clean[keep]) and bool(n[3].isnan().all()) and bool(n[5].isnan().all())
    codes, _ = parts(q)
    assert ((codes[3] & 0x7f) == 0x7f).all() and not ((codes[keep] & 0x7f) == 0x7f).any()


@pytest.mark.gpu
def test_block_norm_rows_of_nothing():
    norm = il.BlockNorm(pre_w=torch.ones(40, device="cuda"), post=True)
    x = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    stats = torch.empty((0, 4), device="cuda")
    il.iris_block_norm(x, norm, y=x, n=torch.empty_like(x), stats=stats)
    sums = {k: torch.full((40,), float("nan"), device="cuda") for k in ("dpre_w", "dpre_b", "dpost_w", "dpost_b")}
    il.iris_block_norm_bwd(None, x, stats, norm, dn=x, y=x, **sums)
    assert all(bool((s == 0).all()) for s in sums.values())
    none = torch.empty((5, 0), dtype=torch.bfloat16, device="cuda")
    il.iris_block_norm(none, il.BlockNorm(), n=torch.empty_like(none))


@pytest.mark.gpu
@pytest.mark.parametrize("gates", [None, 0, 1])
def test_block_norm_bwd_gives_zeros_for_a_gate_without_rows(gates):
    """One gate (a vector, or a matrix of one row) that no row uses has a gradient of
    zeros, as weights have; a gate matrix without rows has none."""
    gate = torch.ones(40 if gates is None else (gates, 40), device="cuda")
    norm = il.BlockNorm(gate=gate, rows_per_gate=None if gates is None else 3)
    x, stats = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 4), device="cuda")
    wide = torch.full((3, 40), float("nan"), device="cuda")
    dgate = wide[1].view(gate.shape) if gate.numel() else wide[1:1]
    il.iris_block_norm_bwd(None, x, stats, norm, dr=x, y=x, dgate=dgate)
    assert bool((dgate == 0).all()) and bool(wide[[0, 2]].isnan().all())
    assert gate.numel() > 0 or bool(wide.isnan().all())


# ---------------------------------------------------------- product, epilogue

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def mm_case(M, N, K, dtype, block, seed):
    A, B = from_gpu(sample(M, K, seed)), il.iris_fp8_empty(N, K, block)
    il.iris_fp8_quantize(torch.from_numpy(sample(N, K, seed + 1, 0.0) / np.sqrt(max(K, 1))).to(torch.float32).cuda(), B)
    a, b = ref.values(*parts(A)), ref.values(*parts(B), block)
    v, size = a @ b.T, np.abs(a) @ np.abs(b).T
    off = (K + 2) * 2.0 ** -23 * size + (0.0 if dtype == "fp32" else 2.0 ** -10) * size
    return A, B, v, off


def check_mm_act(M, N, K, dtype, block, act, p, bias, residual, with_z, out, seed=0, pitch=None, offset=0):
    note(f"mm act {M}x{N}x{K} {dtype} block {block} {act} p {p} bias {bias} residual {residual} z {with_z} out {out}")
    A, B, v, off = mm_case(M, N, K, dtype, block, M + N + K + seed)
    rng = np.random.default_rng(seed + 5)
    bt = None
    if bias:
        bt, bv = on_gpu(rng.normal(size=(1, N)), dtype)
        bt, off, v = bt.reshape(-1), off + 2.0 ** -23 * (np.abs(v) + np.abs(bv)), v + bv
    rt, rv = on_gpu(sample(M, N, seed + 6), dtype, pitch, offset) if residual else (None, 0.0)
    alpha = 0.6 if residual else 1.0
    m = bref.mask(M, N, p, SEED, OFFSET) if p > 0 else 1.0
    c = bref.act(v, act)
    c_off = alpha * m * (1.13 * off + 1e-5 * np.abs(c))
    want = rv + alpha * m * c
    c_off = c_off + 3 * bref.EPS32 * (np.abs(rv) + np.abs(alpha * m * c))
    C, c_in = out_of(M, N, dtype, pitch, offset) if "C" in out else (None, None)
    z, z_in = out_of(M, N, dtype, pitch, offset) if with_z else (None, None)
    q = fresh(M, N) if "q" in out else None
    il.iris_fp8_mm_act(C, A, B, act=act, bias=bt, z=z, residual=rt, alpha=alpha, q=q, dtype=DT[dtype],
                       dropout=il.Dropout(p, SEED, OFFSET) if p > 0 else None)
    if C is not None:
        close(C, want, c_off, dtype, "C")
        assert c_in()
    if z is not None:
        close(z, v, off, dtype, "z")
        assert z_in()
    if q is not None:
        close8(q, want, c_off, "q")


def check_mm_act_bwd(M, N, K, dtype, block, act, p, with_dbias, seed=0, pitch=None, offset=0):
    note(f"mm act backward {M}x{N}x{K} {dtype} block {block} {act} p {p} dbias {with_dbias}")
    A, B, v, off = mm_case(M, N, K, dtype, block, M + N + K + seed + 1)
    z, zv = on_gpu(2 * sample(M, N, seed + 8), dtype, pitch, offset)
    m = (bref.mask(M, N, p, SEED, OFFSET) if p > 0 else 1.0) * 0.9
    s = bref.slope(zv, act)
    want = m * v * s
    c_off = m * (off * np.abs(s) + 1.3e-5 * (np.abs(v) + off)) + 3 * bref.EPS32 * np.abs(want)
    outs = []
    for _ in range(2):
        C, c_in = out_of(M, N, dtype, pitch, offset)
        db = torch.full((N,), float("nan"), dtype=DT[dtype], device="cuda") if with_dbias else None
        il.iris_fp8_mm_act_bwd(C, A, B, z, act, alpha=0.9, dropout=il.Dropout(p, SEED, OFFSET) if p > 0 else None, dbias=db)
        outs.append((C, db))
        assert c_in()
    close(C, want, c_off, dtype, "C")
    assert torch.equal(outs[0][0], outs[1][0])
    if with_dbias:
        close(db, want.sum(0), (c_off + (M + 32) * bref.EPS32 * np.abs(want)).sum(0), dtype, "dbias")
        assert torch.equal(outs[0][1], outs[1][1])


SMALL_MM = [(1, 1, 1), (1, 64, 128), (1, 257, 500), (2, 4096, 256), (7, 1376, 512), (17, 300, 129), (33, 256, 1100), (64, 64, 64),
            (65, 130, 640), (96, 1000, 384), (100, 36, 2000), (128, 128, 128), (200, 1376, 77), (257, 513, 1025)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,block", [("fp16", 128), ("bf16", 1), ("fp32", 128)])
@pytest.mark.parametrize("M,N,K", SMALL_MM)
def test_mm_act(M, N, K, dtype, block):
    for i, act in enumerate(ACTS):
        check_mm_act(M, N, K, dtype, block, act, p=(0.0, 0.3)[i % 2], bias=i % 3 != 0, residual=i % 2 == 0, with_z=i > 1,
                     out=("C", "q", "Cq")[i % 3], seed=i)
    check_mm_act(M, N, K, dtype, block, "gelu", 0.1, True, True, True, "Cq", pitch=N + 5, offset=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,block", [("fp16", 128), ("bf16", 1), ("fp32", 128)])
@pytest.mark.parametrize("M,N,K", SMALL_MM)
def test_mm_act_bwd(M, N, K, dtype, block):
    for i, act in enumerate(ACTS[1:]):
        check_mm_act_bwd(M, N, K, dtype, block, act, p=(0.0, 0.3)[i % 2], with_dbias=i != 2, seed=i)
    check_mm_act_bwd(M, N, K, dtype, block, "silu", 0.1, True, pitch=N + 5, offset=3)


# every tile, whole and with a split contraction
PLANS = [("fp16", 97, 101, 1100, (64, 64, 1)), ("bf16", 301, 397, 4111, (64, 64, 9)), ("bf16", 1501, 2051, 301, (128, 64, 1)),
         ("fp16", 2051, 2053, 311, (128, 128, 1)), ("bf16", 517, 2053, 8305, (128, 128, 3)), ("fp16", 3005, 4103, 305, (256, 256, 1)),
         ("fp32", 301, 397, 4111, (64, 64, 9)), ("fp32", 1503, 1505, 301, (128, 64, 1)), ("fp32", 2051, 2053, 311, (128, 128, 1)),
         ("fp32", 3005, 5003, 305, (256, 256, 1))]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,N,K,want", PLANS)
def test_mm_act_of_each_plan(dtype, M, N, K, want):
    if M < 1000:
        assert plan(M, N, K, dtype) == want
    check_mm_act(M, N, K, dtype, 1, "gelu_tanh", 0.2, True, True, True, "C", pitch=N + 3, offset=1)
    check_mm_act(M, N, K, dtype, 128, "silu", 0.0, True, False, False, "q")
    check_mm_act_bwd(M, N, K, dtype, 128, "gelu", 0.2, True)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(3, 40), (70, 90), (200, 130), (700, 1100), (2300, 2100)])
def test_mm_act_of_nothing(M, N):
    """K = 0 gives act(bias); no rows give a bias gradient of zeros."""
    A, B = il.iris_fp8_empty(M, 0), il.iris_fp8_empty(N, 0)
    bt, bv = on_gpu(np.random.default_rng(1).normal(size=(1, N)), "fp32")
    C, q = torch.full((M, N), float("nan"), device="cuda"), fresh(M, N)
    il.iris_fp8_mm_act(C, A, B, act="silu", bias=bt.reshape(-1), q=q)
    want = np.broadcast_to(bref.act(bv, "silu"), (M, N))
    close(C, want, 1e-5 * np.abs(want), "fp32", "C")
    close8(q, want, 1e-5 * np.abs(want), "q")
    db = torch.full((N,), float("nan"), device="cuda")
    z0 = torch.empty((0, N), device="cuda")
    il.iris_fp8_mm_act_bwd(torch.empty_like(z0), il.iris_fp8_empty(0, 64), il.iris_fp8_empty(N, 64), z0, "relu", dbias=db)
    assert bool((db == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_far_out(act):
    """Values to the ends of the range through a product of one column: finite where the function is."""
    z = np.array([0.0, -0.0, 1e-30, -1e-30, 1.0, -1.0, 5.0, -5.0, 8.0, -8.0, 12.0, -12.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4,
                  1e15, -1e15, 1e30, -1e30, 3e38, -3e38])
    n = len(z)
    bt, zv = on_gpu(z.reshape(1, n), "fp32")
    for M in (2, 200):
        A, B = il.iris_fp8_empty(M, 0), il.iris_fp8_empty(n, 0)
        C = torch.full((M, n), float("nan"), device="cuda")
        il.iris_fp8_mm_act(C, A, B, act=act, bias=bt.reshape(-1))
        with np.errstate(over="ignore", invalid="ignore"):
            want = np.where(np.abs(zv) > 1e3, np.maximum(zv, 0.0), bref.act(np.clip(zv, -1e3, 1e3), act))
            slope = np.where(np.abs(zv) > 1e3, (zv > 0) * 1.0, bref.slope(np.clip(zv, -1e3, 1e3), act))
        got = values(C)
        # subnormal results may be flushed
        assert np.all(np.abs(got - want) <= 2e-5 * np.abs(want) + 2.0 ** -126), (got[0], want)
        ones, one = torch.ones((M, 1), device="cuda"), torch.ones((n, 1), device="cuda")
        A, B = il.iris_fp8_empty(M, 1), il.iris_fp8_empty(n, 1)
        il.iris_fp8_quantize(ones, A)
        il.iris_fp8_quantize(one, B)
        il.iris_fp8_mm_act_bwd(C, A, B, bt.expand(M, n).contiguous(), act)
        assert np.all(np.abs(values(C) - slope) <= 2e-5), (values(C)[0], slope)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 90, 300])
def test_mm_act_nan_stays_in_its_row(M):
    A, B, v, _ = mm_case(M, 200, 300, "bf16", 128, 3)
    C, clean = (torch.empty((M, 200), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = fresh(M, 200)
    for act in ACTS:
        codes = A.codes.view(torch.uint8)
        kept = int(codes[1, 17])
        il.iris_fp8_mm_act(clean, A, B, act=act)
        codes[1, 17] = 0x7F
        il.iris_fp8_mm_act(C, A, B, act=act, q=q)
        codes[1, 17] = kept
        rest = [i for i in range(M) if i != 1]
        assert bool(C[1].isnan().all()) and torch.equal(C[rest], clean[rest])
        c8, _ = parts(q)
        assert ((c8[1] & 0x7F) == 0x7F).all() and not ((c8[rest] & 0x7F) == 0x7F).any()


# ------------------------------------------------- streams, graphs, threads

def block_step():
    """Closures of the operators that use the library's workspace, with fixed inputs, and their outputs."""
    t, v, plain, norm, group, stream = norm_case(600, 1376, NORM_WAYS[0], "bf16", 3)
    stats = torch.empty((600, 4), device="cuda")
    r = torch.empty((600, 1376), device="cuda")
    n = torch.empty((600, 1376), dtype=torch.bfloat16, device="cuda")
    out = {"r": r, "n": n, "stats": stats, "dx": torch.empty_like(r), "dy": torch.empty_like(n),
           **{k: torch.empty(1376, device="cuda") for k in ("dpre_w", "dpost_w", "dgate")}}
    A, B, _, _ = mm_case(301, 397, 4111, "bf16", 128, 5)
    z = torch.randn((301, 397), device="cuda").to(torch.bfloat16)
    out |= {"C": torch.empty_like(z), "dbias": torch.empty(397, dtype=torch.bfloat16, device="cuda"), "D": torch.empty_like(z)}
    few, wide = mm_case(33, 1000, 512, "bf16", 128, 6)[:2]
    q = fresh(33, 1000)
    out["codes"] = q.codes.view(torch.uint8)
    drop = il.Dropout(0.2, 1, 2)
    out |= {"dropped": torch.empty_like(n), "sums": torch.empty(1376, dtype=torch.bfloat16, device="cuda")}

    def run():
        il.iris_dropout(out["dropped"], t["y"], drop, sums=out["sums"])
        il.iris_block_norm(t["x"], norm, y=t["y"], r=r, n=n, stats=stats)
        il.iris_block_norm_bwd(out["dx"], r, stats, norm, dn=n, dr=r, y=t["y"], dy=out["dy"], dpre_w=out["dpre_w"],
                               dpost_w=out["dpost_w"], dgate=out["dgate"])
        il.iris_fp8_mm_act_bwd(out["C"], A, B, z, "silu", dropout=drop, dbias=out["dbias"])
        il.iris_fp8_mm_act(out["D"], A, B, act="gelu", residual=z)
        il.iris_fp8_mm_act(None, few, wide, act="relu", q=q, dtype=torch.bfloat16)
    return run, out


def clear(out):
    for t in out.values():
        t.zero_()


@pytest.mark.gpu
def test_other_stream_and_graph_replay():
    note("block operators on another stream and in a graph")
    run, out = block_step()
    run()
    torch.cuda.synchronize()
    want = {k: t.clone() for k, t in out.items()}
    clear(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
    for _ in range(3):
        clear(out)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), k
        clear(out)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)


@pytest.mark.gpu
def test_threads_that_share_a_stream():
    """Two launches of one call are enqueued together: threads on one stream do not mix their sums."""
    note("block operators from threads")
    made = [block_step() for _ in range(3)]
    for run, out in made:
        run()
    torch.cuda.synchronize()
    want = [{k: t.clone() for k, t in out.items()} for _, out in made]
    errors = []

    def work(run):
        try:
            for _ in range(20):
                run()
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    ts = [threading.Thread(target=work, args=(run,)) for run, _ in made]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for (_, out), w in zip(made, want):
        assert all(torch.equal(out[k], w[k]) for k in w)


@pytest.mark.gpu
def test_callers_workspaces():
    rows, cols = 600, 1376
    need = il.iris_block_norm_bwd_workspace_size(rows, cols)
    t, v, plain, norm, group, stream = norm_case(rows, cols, NORM_WAYS[0], "bf16", 3)
    got = run_bwd(t, v, plain, norm, group, stream, "bf16", rows, cols)
    assert need > 0 and got
    stats = torch.ones((rows, 4), device="cuda")
    two = [torch.empty(cols, device="cuda") for _ in range(2)]
    il.iris_block_norm_bwd(None, t["x"], stats, norm, dn=t["y"], y=t["y"], dpre_w=two[0])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    il.iris_block_norm_bwd(None, t["x"], stats, norm, dn=t["y"], y=t["y"], dpre_w=two[1], workspace=ws)
    assert torch.equal(*two)
    with pytest.raises(il.IrisError, match="smaller"):
        il.iris_block_norm_bwd(None, t["x"], stats, norm, dn=t["y"], y=t["y"], dpre_w=two[1], workspace=ws[:-256])
    for M, N, K in ((301, 397, 4111), (33, 397, 512), (300, 300, 300)):
        A, B, _, _ = mm_case(M, N, K, "bf16", 128, 5)
        z = torch.randn((M, N), device="cuda").to(torch.bfloat16)
        C = [torch.empty_like(z) for _ in range(2)]
        db = [torch.empty(N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        need = il.iris_fp8_mm_act_workspace_size(M, N, K, torch.bfloat16, dbias=True)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        for c, d, w in zip(C, db, (None, ws)):
            il.iris_fp8_mm_act_bwd(c, A, B, z, "silu", dbias=d, workspace=w)
        assert torch.equal(*C) and torch.equal(*db)
        with pytest.raises(il.IrisError, match="smaller"):
            il.iris_fp8_mm_act_bwd(C[0], A, B, z, "silu", dbias=db[0], workspace=ws[:-256])


@pytest.mark.gpu
def test_masks_of_the_operators_are_one():
    """What the product's epilogue drops, iris_dropout drops, and so does the norm's residual sum."""
    M, N = 70, 1030
    d = il.Dropout(0.4, 11, 12)
    ones = torch.ones((M, N), device="cuda")
    a = torch.empty_like(ones)
    il.iris_dropout(a, ones, d)
    r = torch.empty_like(ones)
    il.iris_block_norm(torch.zeros_like(ones), il.BlockNorm(dropout=d), y=ones.to(torch.bfloat16), r=r)
    assert torch.equal(a, r)
    bias = torch.ones(N, device="cuda")
    for rows in (M, 300):
        c = torch.empty((rows, N), device="cuda")
        il.iris_fp8_mm_act(c, il.iris_fp8_empty(rows, 0), il.iris_fp8_empty(N, 0), bias=bias, dropout=d)
        assert torch.equal(c[:M], a)
