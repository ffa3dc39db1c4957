"""The 8-bit operators on the GPU against the plain 64-bit forms of fp8_ref.

Quantising given values has one right answer, so codes and scales are compared
bit for bit. Products: any order of a 32-bit sum of n terms is within
n 2^-23 sum |a b| of the exact one (an ulp, not half of one, for every addition,
in case the matrix unit truncates inside), then one rounding to C's type. For a
16-bit C the matrix unit drops what is under 2^-13 of the largest of 8 products
that it adds: at most 8 * 2^-13 of that product for each 8, 2^-10 sum |a b| in
all. Sums of small integers are exact. Computed activations: the value before its
8-bit rounding is good to 1e-5 (the hardware's exp2 and reciprocal), its code
to half an e4m3 step more.
"""
import threading

import numpy as np
import pytest
import torch

import fp8_ref as ref
import gemm_collective_tile_amd as il
from fp8_plan import OF_EACH_PLAN, plan
from gpu_util import note

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ULP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def u8(t):
    return t.detach().contiguous().view(torch.uint8).cpu().numpy()


def parts(q):
    return u8(q.codes), u8(q.scales)


def fresh(rows, cols, block=1):
    """An output whose memory is filled with a pattern, so that what is not written shows."""
    q = il.iris_fp8_empty(rows, cols, block)
    for t in (q.codes, q.scales):
        whole = torch.as_strided(t.view(torch.uint8), (t.shape[0], t.stride(0)), (t.stride(0), 1))
        whole.fill_(0xA5)
    return q


def assert_untouched(q, what):
    for t in (q.codes, q.scales):
        whole = torch.as_strided(t.view(torch.uint8), (t.shape[0], t.stride(0)), (t.stride(0), 1)).cpu()
        assert bool((whole[:, t.shape[1]:] == 0xA5).all()), f"{what}: bytes past the last column were written"


def made(x, block=1):
    """An Fp8 operand of the values x, made by the plain form; its padding holds NaN codes."""
    codes, scales = ref.quantize(x, block)
    return put(codes, scales, block)


def put(codes, scales, block=1):
    q = il.iris_fp8_empty(codes.shape[0], codes.shape[1], block)
    for t, src, pad in ((q.codes, codes, 0x7f), (q.scales, scales, 0xff)):
        if t.numel() == 0:
            continue
        whole = torch.as_strided(t.view(torch.uint8), (t.shape[0], t.stride(0)), (t.stride(0), 1))
        whole.fill_(pad)
        whole[:, :t.shape[1]] = torch.from_numpy(src.copy())
    return q


def sample(rows, cols, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) * np.exp2(rng.normal(size=(rows, 1)) * spread)
    x[:, rng.random(cols) < 0.02] *= 20
    if rows > 3:
        x[2] = 0.0
    return x


def on_gpu(x, dtype, pitch=None, offset=0):
    """x rounded to dtype on the GPU, at a row pitch and an element offset; and its float64 values."""
    t = torch.from_numpy(x).to(torch.float32).to(DT[dtype])
    rows, cols = t.shape
    pitch = cols if pitch is None else pitch
    store = torch.full((offset + rows * pitch + 8,), float("nan"), dtype=DT[dtype], device="cuda")
    v = torch.as_strided(store, (rows, cols), (pitch, 1), offset)
    v.copy_(t)
    return v, t.double().numpy()


def check_quantized(q, x, block, what):
    codes, scales = parts(q)
    wc, ws = ref.quantize(x, block)
    assert np.array_equal(scales, ws), f"{what}: scales differ at {np.argwhere(scales != ws)[:4].tolist()}"
    nan = (wc & 0x7f) == 0x7f
    assert np.array_equal((codes & 0x7f) == 0x7f, nan), f"{what}: NaN codes differ"
    bad = (codes != wc) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} codes differ, first at {np.argwhere(bad)[0].tolist()}"
    assert_untouched(q, what)


SHAPES = [(1, 1), (1, 128), (1, 4096), (3, 127), (5, 129), (128, 128), (129, 257), (200, 1376), (33, 15), (257, 16),
          (1000, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype):
    x, xv = on_gpu(sample(rows, cols, rows * 7919 + cols), dtype)
    for block in (1, 128):
        note(f"quantize {rows}x{cols} {dtype} block {block}")
        q, qt = fresh(rows, cols, block), fresh(cols, rows, block)
        il.iris_fp8_quantize(x, q, qt)
        check_quantized(q, xv, block, "rows of both")
        check_quantized(qt, np.ascontiguousarray(xv.T), block, "columns of both")
        q, qt = fresh(rows, cols, block), fresh(cols, rows, block)
        il.iris_fp8_quantize(x, q)
        il.iris_fp8_quantize(x, None, qt)
        check_quantized(q, xv, block, "rows")
        check_quantized(qt, np.ascontiguousarray(xv.T), block, "columns")


@pytest.mark.gpu
@pytest.mark.parametrize("pitch,offset", [(320, 0), (304, 8), (301, 0), (300, 1), (303, 5)])
def test_quantize_pitch_and_offset(pitch, offset):
    for dtype in DT:
        x, xv = on_gpu(sample(70, 300, pitch), dtype, pitch, offset)
        note(f"quantize 70x300 {dtype} pitch {pitch} offset {offset}")
        q, qt = fresh(70, 300), fresh(300, 70)
        il.iris_fp8_quantize(x, q)
        check_quantized(q, xv, 1, "rows")
        il.iris_fp8_quantize(x, q, qt)
        check_quantized(q, xv, 1, "rows of both")
        check_quantized(qt, np.ascontiguousarray(xv.T), 1, "columns")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [1, 7, 8, 9, 15, 17, 30, 31, 113, 121, 127, 129, 143])
def test_quantize_ragged_rows_keep_their_neighbours_out(cols, dtype):
    """A ragged piece may be read with what follows its row, which has no say in the
    row's scale or codes: rows alternate between ordinary and 1000 times larger values."""
    for rows, pitch, offset in ((1, cols, 1), (2, cols, 0), (131, cols, 0), (131, cols + 3, 1), (130, cols + 16, 2)):
        note(f"quantize ragged {rows}x{cols} {dtype} pitch {pitch} offset {offset}")
        v = sample(rows, cols, cols * 31 + rows)
        v[1::2] *= 1000.0
        x, xv = on_gpu(v, dtype, pitch, offset)
        q, qt = fresh(rows, cols), fresh(cols, rows)
        il.iris_fp8_quantize(x, q)
        check_quantized(q, xv, 1, "rows")
        q = fresh(rows, cols)
        il.iris_fp8_quantize(x, q, qt)
        check_quantized(q, xv, 1, "rows of both")
        check_quantized(qt, np.ascontiguousarray(xv.T), 1, "columns")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_special_values(dtype):
    """Infinities, NaN, blocks of nothing else, zeros of both signs, the largest and the smallest values, ties."""
    top = float(torch.finfo(DT[dtype]).max)
    low = float(torch.finfo(DT[dtype]).smallest_normal)
    x = sample(140, 520, 5)
    x[0, 3], x[1, 130], x[3, 200] = np.inf, -np.inf, np.nan
    x[4, 128:256] = np.nan
    x[5, :128] = -0.0
    x[6, :256] = top
    x[7, :256] = low / 2          # subnormal in its type
    x[8, :128] = low
    x[9, :128] = 448.0 * np.exp2(np.arange(128) % 3 - 1)
    x[10, :128] = 448.0
    x[11, :128] = 449.0
    x[12, :127] = (ref.TABLE[:126] + ref.TABLE[1:127])[np.arange(127) % 126] / 2   # midpoints
    x[12, 127] = 448.0
    x[:, 400] = np.inf
    x[:, 401] = np.nan
    xg, xv = on_gpu(x, dtype)
    note(f"quantize special values {dtype}")
    for block in (1, 128):
        q, qt = fresh(140, 520, block), fresh(520, 140, block)
        il.iris_fp8_quantize(xg, q, qt)
        check_quantized(q, xv, block, "rows")
        check_quantized(qt, np.ascontiguousarray(xv.T), block, "columns")
        if block == 1:
            il.iris_fp8_quantize(xg, q)
            check_quantized(q, xv, 1, "rows alone")


SIGNALLING = {"fp16": 0x7c01, "bf16": 0x7f81, "fp32": 0x7f800001}


def with_nan_beside_the_largest(dtype, rows, cols, places):
    """Ordinary values with, for every (row, column, other column) of `places`, a signalling NaN and, at the other
    column, a value that is the largest of all its blocks; on the GPU, and in float64."""
    v = sample(rows, cols, 11, 0.0)
    for n, (r, c, o) in enumerate(places):
        v[r, o] = 3000.0 + n
    x, _ = on_gpu(v, dtype)
    bits = x.view(torch.int32 if dtype == "fp32" else torch.int16)
    sign = 1 << (31 if dtype == "fp32" else 15)
    for n, (r, c, o) in enumerate(places):
        bits[r, c] = SIGNALLING[dtype] - (sign if n % 2 else 0)    # both signs
    values = x.double().cpu().numpy()
    assert np.isnan(values).sum() == len(places)
    return x, values


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_signalling_nan_leaves_the_scale(dtype):
    """A signalling NaN at every place of a piece, its neighbours in the hardware's pairs the largest of their blocks."""
    for cols in (256, 253):
        note(f"quantize signalling NaN {dtype} {cols}")
        diagonal = [(p, p, p ^ 1) for p in range(128)] + [(p, 128 + p, 128 + (p + 1) % 125) for p in range(0, 125, 2)]
        x, xv = with_nan_beside_the_largest(dtype, 128, cols, diagonal)
        q, qt = fresh(128, cols), fresh(cols, 128)
        il.iris_fp8_quantize(x, q)
        check_quantized(q, xv, 1, "rows")
        q = fresh(128, cols)
        il.iris_fp8_quantize(x, q, qt)
        check_quantized(q, xv, 1, "rows of both")
        check_quantized(qt, np.ascontiguousarray(xv.T), 1, "columns")
    places = [(128 * i + 3 * i + j, 128 * j + 8 * i + 2 * j + i % 2, 128 * j + (8 * i + 2 * j + i % 2 ^ 1))
              for i in range(4) for j in range(4)]
    x, xv = with_nan_beside_the_largest(dtype, 512, 512, places)
    q, qt = fresh(512, 512, 128), fresh(512, 512, 128)
    il.iris_fp8_quantize(x, q, qt)
    check_quantized(q, xv, 128, "blocks")
    check_quantized(qt, np.ascontiguousarray(xv.T), 128, "blocks of columns")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_swiglu_signalling_nan_leaves_the_scale(dtype):
    diagonal = [(p, p, p ^ 1) for p in range(128)]
    note(f"swiglu signalling NaN {dtype}")
    gate, gv = with_nan_beside_the_largest(dtype, 128, 128, diagonal)
    up, uv = with_nan_beside_the_largest(dtype, 128, 128, [(p, p ^ 3, p ^ 2) for p in range(128)])
    h, gk, uk = (fresh(128, 128) for _ in range(3))
    il.iris_fp8_swiglu(h, gate, up, gk, uk)
    check_quantized(gk, gv, 1, "gate")
    check_quantized(uk, uv, 1, "up")
    assert np.array_equal((parts(h)[0] & 0x7f) == 0x7f, np.isnan(gv) | np.isnan(uv))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_kept(rows, cols):
    """An 8-bit matrix turned around: its values are given, so the new codes and scales have one right answer."""
    rng = np.random.default_rng(rows + cols)
    codes = rng.integers(0, 256, (rows, cols)).astype(np.uint8)
    if rows < 8:
        codes[(codes & 0x7f) == 0x7f] = 0
    scales = rng.integers(100, 140, (rows, -(-cols // 128))).astype(np.uint8)
    scales[0] = 1
    note(f"quantize kept {rows}x{cols}")
    qt = fresh(cols, rows)
    il.iris_fp8_quantize(put(codes, scales), None, qt)
    check_quantized(qt, np.ascontiguousarray(ref.values(codes, scales).T), 1, "columns")


# ------------------------------------------------------------------ products

def check_product(C, a, b, bias, old, dtype, what):
    exact = a @ b.T
    size = np.abs(a) @ np.abs(b).T
    if bias is not None:
        exact, size = exact + bias, size + np.abs(bias)
    if old is not None:
        exact, size = exact + old, size + np.abs(old)
    got = C.double().cpu().numpy()
    bound = (a.shape[1] + 2) * 2.0 ** -23 * size + ULP[dtype] * np.abs(exact) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    bound = bound + (0.0 if dtype == "fp32" else 2.0 ** -10) * size
    off = ~(np.abs(got - exact) <= bound)
    assert not off.any(), (what, int(off.sum()), np.argwhere(off)[0].tolist(), got[off][0], exact[off][0])


MM_SHAPES = [(1, 1, 1), (1, 64, 128), (1, 257, 500), (2, 4096, 256), (3, 100, 130), (7, 1376, 4096), (16, 128, 1024),
             (17, 300, 129), (33, 256, 11008), (64, 64, 64), (65, 130, 640), (100, 36, 2000), (127, 255, 127),
             (128, 128, 128), (129, 257, 385), (200, 1376, 777), (256, 256, 1152), (257, 513, 1025), (300, 1000, 96),
             (513, 768, 512), (1030, 2050, 390)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", MM_SHAPES)
def test_mm(M, N, K):
    for dtype, block, with_bias in (("fp16", 128, True), ("bf16", 1, False), ("fp32", 1, True), ("fp32", 128, False)):
        note(f"mm {M}x{N}x{K} {dtype} block {block} bias {with_bias}")
        A, B = made(sample(M, K, M + K)), made(sample(N, K, N + K + 1, 0.0) / np.sqrt(K), block)
        a, b = ref.values(*parts(A)), ref.values(*parts(B), block)
        bias, bv = on_gpu(np.random.default_rng(N).normal(size=(1, N)), dtype) if with_bias else (None, None)
        C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
        il.iris_fp8_mm(C, A, B, None if bias is None else bias.reshape(-1))
        check_product(C, a, b, bv, None, dtype, (M, N, K, dtype, block))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,block", [("fp16", 128), ("bf16", 1), ("fp32", 1)])
@pytest.mark.parametrize("M,N,K", [(3900, 4000, 2100), (1900, 2100, 1500), (1000, 1300, 2000), (500, 1000, 700)])
def test_mm_of_each_tile(M, N, K, dtype, block):
    """Sizes that the plan gives 256 x 256, 128 x 128, 128 x 64 and 64 x 64 tiles, ragged in all three lengths."""
    note(f"mm tiles {M}x{N}x{K} {dtype}")
    A, B = made(sample(M, K, 1)), made(sample(N, K, 2, 0.0) / np.sqrt(K), block)
    a, b = ref.values(*parts(A)), ref.values(*parts(B), block)
    C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
    il.iris_fp8_mm(C, A, B)
    check_product(C, a, b, None, None, dtype, (M, N, K, dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,N,K,want", OF_EACH_PLAN)
def test_mm_of_each_plan(dtype, M, N, K, want):
    """Every tile, whole and with a split contraction: with a bias along N into whole rows, then along M and added to
    what an unaligned C of odd pitch holds; both twice, with the same bits."""
    assert plan(M, N, K, dtype) == want
    note(f"mm plan {M}x{N}x{K} {dtype} {want}")
    block = 128 if K % 2 else 1
    A, B = from_gpu(sample(M, K, 1)), il.iris_fp8_empty(N, K, block)
    il.iris_fp8_quantize(torch.from_numpy(sample(N, K, 2, 0.0) / np.sqrt(K)).to(torch.float32).cuda(), B)
    a, b = ref.values(*parts(A)), ref.values(*parts(B), block)
    exact, size = a @ b.T, np.abs(a) @ np.abs(b).T

    def check(C, more, old, what):
        e, s = exact + more + old, size + np.abs(more) + np.abs(old)
        bound = (K + 2) * 2.0 ** -23 * s + ULP[dtype] * np.abs(e) + (0.0 if dtype == "fp32" else 2.0 ** -10) * s
        off = ~(np.abs(C.double().cpu().numpy() - e) <= bound + (2.0 ** -25 if dtype == "fp16" else 0.0))
        assert not off.any(), (what, int(off.sum()), np.argwhere(off)[0].tolist())
    along_n, nv = on_gpu(np.random.default_rng(3).normal(size=(1, N)), dtype)
    C, D = (torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    for out in (C, D):
        il.iris_fp8_mm(out, A, B, along_n.reshape(-1))
    check(C, nv, 0.0, "bias along N")
    assert torch.equal(C, D)
    along_m, mv = on_gpu(np.random.default_rng(4).normal(size=(M, 1)), dtype)
    first = None
    for _ in range(2):
        old, ov = on_gpu(sample(M, N, 5), dtype, N + 5, 3)
        il.iris_fp8_mm(old, A, B, along_m.reshape(-1), accumulate=True, config=il.Config(flags=il.IRIS_FLAG_BIAS_ALONG_M))
        if first is None:
            first = old
            check(old, mv, ov, "accumulated, bias along M")
    assert torch.equal(first, old)
    outside = torch.empty(0, dtype=DT[dtype], device="cuda").set_(old.untyped_storage()).clone()
    torch.as_strided(outside, (M, N), (N + 5, 1), 3).fill_(float("nan"))
    assert bool(outside.isnan().all()), "C's padding was written"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,block", [("fp16", 128), ("bf16", 1), ("fp32", 128)])
@pytest.mark.parametrize("M", [1, 20, 48, 63, 66, 90])
def test_mm_of_few_rows_and_many_columns(M, dtype, block):
    """One, two and three blocks of 16 columns a workgroup, ragged in all lengths;
    up to 64 rows a column's result is the same whatever the number of columns."""
    for N, K in ((300, 1100), (4101, 1100), (8205, 1100), (8205, 129), (4101, 100)):
        note(f"mm few rows {M}x{N}x{K} {dtype}")
        A, B = made(sample(M, K, 1)), made(sample(N, K, 2, 0.0) / np.sqrt(K), block)
        a, b = ref.values(*parts(A)), ref.values(*parts(B), block)
        C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
        il.iris_fp8_mm(C, A, B)
        check_product(C, a, b, None, None, dtype, (M, N, K, dtype))
        if K == 1100 and M <= 64:
            part = il.Fp8(B.codes[:256], B.scales[:256 if block == 1 else 2], block)
            D = torch.empty((M, 256), dtype=DT[dtype], device="cuda")
            il.iris_fp8_mm(D, A, part)
            assert torch.equal(C[:, :256], D)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,block", [("fp16", 128), ("bf16", 1), ("fp32", 1)])
@pytest.mark.parametrize("M,N,K", [(2100, 2010, 300), (2054, 1936, 333), (857, 304, 4496), (130, 1000, 21000)])
def test_mm_of_more_tiles_than_units_and_of_splits(M, N, K, dtype, block):
    """128 x 128 tiles, two and four tiles a compute unit, and contractions in several parts."""
    note(f"mm rounds {M}x{N}x{K} {dtype}")
    A, B = made(sample(M, K, 1)), made(sample(N, K, 2, 0.0) / np.sqrt(K), block)
    a, b = ref.values(*parts(A)), ref.values(*parts(B), block)
    C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
    il.iris_fp8_mm(C, A, B)
    check_product(C, a, b, None, None, dtype, (M, N, K, dtype))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Matrices of more than 4 GiB: their last rows are what the same rows alone give."""
    rows, cols = 270_000, 16_384                      # 4.4e9 values
    note("offsets past 32 bits: quantize")
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[:1000].normal_()
    x[-1000:].normal_()
    x[1000:-1000] = 0.5
    q, qt = il.iris_fp8_empty(rows, cols), il.iris_fp8_empty(cols, rows)
    il.iris_fp8_quantize(x, q, qt)
    last = 304                                        # from a multiple of 128 on
    start = rows - last
    start -= start % 128
    p, pt = il.iris_fp8_empty(rows - start, cols), il.iris_fp8_empty(cols, rows - start)
    il.iris_fp8_quantize(x[start:], p, pt)
    for big, small in ((q.codes[start:], p.codes), (q.scales[start:], p.scales), (qt.codes[:, start:], pt.codes),
                       (qt.scales[:, start // 128:], pt.scales)):
        assert torch.equal(big.contiguous().view(torch.uint8), small.contiguous().view(torch.uint8))
    del qt, pt, x
    note("offsets past 32 bits: mm")
    B = made(sample(72, cols, 2) / 128, 128)
    C, tail = (torch.empty((n, 72), dtype=torch.float16, device="cuda") for n in (rows, rows - start))
    il.iris_fp8_mm(C, q, B)
    il.iris_fp8_mm(tail, p, B)
    check = C[start:].float()
    assert torch.allclose(check, tail.float(), rtol=2.0 ** -9, atol=2.0 ** -9 * float(check.abs().max()))
    few = torch.empty((40, rows), dtype=torch.bfloat16, device="cuda")
    part = torch.empty((40, rows - start), dtype=torch.bfloat16, device="cuda")
    a = made(sample(40, cols, 3))
    il.iris_fp8_mm(few, a, q)                         # as the many rows of B
    il.iris_fp8_mm(part, a, p)
    assert torch.equal(few[:, start:], part)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 300, 257), (20, 130, 520), (70, 200, 300), (260, 390, 260), (600, 512, 384)])
def test_mm_accumulate_bias_along_m_and_pitch(M, N, K):
    for dtype in DT:
        for pitch, offset in ((N, 0), (N + 5, 3), (-(-N // 16) * 16 + 16, 0)):
            note(f"mm accumulate {M}x{N}x{K} {dtype} pitch {pitch} offset {offset}")
            A, B = made(sample(M, K, 1)), made(sample(N, K, 2, 0.0) / np.sqrt(K), 128)
            a, b = ref.values(*parts(A)), ref.values(*parts(B), 128)
            old, ov = on_gpu(sample(M, N, 3), dtype, pitch, offset)
            bias, bv = on_gpu(np.random.default_rng(4).normal(size=(M, 1)), dtype)
            store = old.untyped_storage()
            before = torch.empty(0, dtype=DT[dtype], device="cuda").set_(store).clone()
            il.iris_fp8_mm(old, A, B, bias.reshape(-1), accumulate=True,
                           config=il.Config(flags=il.IRIS_FLAG_BIAS_ALONG_M))
            check_product(old, a, b, bv, ov, dtype, (M, N, K, dtype, pitch))
            after = torch.empty(0, dtype=DT[dtype], device="cuda").set_(store)
            outside = torch.ones_like(after, dtype=torch.bool)
            torch.as_strided(outside, (M, N), (pitch, 1), offset).fill_(False)
            assert bool((after[outside].isnan() & before[outside].isnan()).all()), "C's padding was written"


@pytest.mark.gpu
def test_mm_accumulates_by_argument_and_by_flag():
    note("mm accumulate by flag")
    A, B = made(sample(70, 260, 1)), made(sample(90, 260, 2))
    outs = []
    for kw in (dict(accumulate=True), dict(config=il.Config(flags=il.IRIS_FLAG_ACCUMULATE)),
               dict(config={"flags": il.IRIS_FLAG_ACCUMULATE})):
        C = torch.full((70, 90), 3.0, dtype=torch.float32, device="cuda")
        il.iris_fp8_mm(C, A, B, **kw)
        outs.append(C)
    plain = torch.empty_like(outs[0])
    il.iris_fp8_mm(plain, A, B)
    assert torch.equal(outs[0], plain + 3.0)
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 384, 4096), (5, 200, 11008), (48, 256, 2000), (130, 140, 1500), (520, 300, 4000)])
def test_mm_integers_are_exact(M, N, K):
    """Small integers times powers of two: every partial sum fits 24 bits, so fp32 results are exact."""
    rng = np.random.default_rng(K)
    a, b = rng.integers(-8, 9, (M, K)).astype(np.float64), rng.integers(-8, 9, (N, K)).astype(np.float64)
    sa = np.full((M, -(-K // 128)), 127, np.uint8) + (np.arange(M)[:, None] % 3).astype(np.uint8)
    sb = np.full((N, -(-K // 128)), 127, np.uint8) - (np.arange(N)[:, None] % 3).astype(np.uint8)
    note(f"mm integers {M}x{N}x{K}")
    C = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    il.iris_fp8_mm(C, put(ref.encode(a), sa), put(ref.encode(b), sb))
    want = (a * np.exp2(np.arange(M) % 3)[:, None]) @ (b * np.exp2(-(np.arange(N) % 3.0))[:, None]).T
    assert np.array_equal(C.double().cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_mm_block_scales_act_per_block(M):
    """Ones everywhere: an output is the sum over k blocks of the two scales times the block's length."""
    N, K = 270, 128 * 9 + 40
    rng = np.random.default_rng(M)
    sa = rng.integers(124, 131, (M, 10)).astype(np.uint8)
    sb = rng.integers(124, 131, (3, 10)).astype(np.uint8)
    one = ref.encode(np.ones((1, 1)))[0, 0]
    length = np.full(10, 128.0)
    length[9] = 40
    for block, s in ((128, sb), (1, rng.integers(124, 131, (N, 10)).astype(np.uint8))):
        note(f"mm block scales M {M} block {block}")
        C = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
        il.iris_fp8_mm(C, put(np.full((M, K), one), sa), put(np.full((N, K), one), s, block))
        wide = np.exp2(s.astype(np.float64) - 127).repeat(block, 0)[:N]
        want = (np.exp2(sa.astype(np.float64) - 127) * length) @ wide.T
        assert np.array_equal(C.double().cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 40, 90, 200])
def test_mm_scale_bytes_of_the_whole_range(M):
    """Scale bytes of one operand from the smallest to the largest against the other's opposite: every one from 1 to
    254 into 16 bits, 3 to 246 (entries that bf16 holds) into 32."""
    N, K = 70, 300
    rng = np.random.default_rng(M)
    a, b = (rng.integers(0, 256, (n, K)).astype(np.uint8) for n in (M, N))
    for codes in (a, b):
        codes[(codes & 0x7f) == 0x7f] = 1
        codes[1], codes[2], codes[3] = 1, rng.integers(1, 8, K), 0x7e    # the smallest, subnormal ones, the largest
    for dtype, lo, hi in (("bf16", 1, 254), ("fp32", 3, 246)):
        for s in sorted({lo, lo + 1, 3, 9, 10, 60, 127, 200, 246, hi}):
            t = max(lo, min(hi, 254 - s))
            note(f"mm scale bytes M {M} {dtype} {s} {t}")
            for sa, sb in ((s, t), (t, s)):
                A, B = put(a, np.full((M, 3), sa, np.uint8)), put(b, np.full((N, 3), sb, np.uint8))
                C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
                il.iris_fp8_mm(C, A, B)
                check_product(C, ref.values(*parts(A)), ref.values(*parts(B)), None, None, dtype, (M, dtype, sa, sb))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 200), (40, 200), (300, 200)])
def test_mm_nan_stays_in_its_row_and_column(M, N):
    K = 520
    note(f"mm nan {M}x{N}")
    ac, asc = ref.quantize(sample(M, K, 1))
    bc, bsc = ref.quantize(sample(N, K, 2))
    ac[M // 2, 515] = 0x7f
    bc[7, 3] = 0xff
    C = torch.zeros((M, N), dtype=torch.float16, device="cuda")
    il.iris_fp8_mm(C, put(ac, asc), put(bc, bsc))
    nan = np.zeros((M, N), bool)
    nan[M // 2] = True
    nan[:, 7] = True
    assert np.array_equal(C.isnan().cpu().numpy(), nan)


@pytest.mark.gpu
def test_mm_lengths_of_zero():
    B = il.iris_fp8_empty(40, 0)
    C = torch.full((3, 40), float("nan"), dtype=torch.float32, device="cuda")
    bias = torch.arange(40, dtype=torch.float32, device="cuda")
    il.iris_fp8_mm(C, il.iris_fp8_empty(3, 0), B, bias)
    assert torch.equal(C, bias.expand(3, 40))
    il.iris_fp8_mm(C, il.iris_fp8_empty(3, 0), B, bias, accumulate=True)
    assert torch.equal(C, 2 * bias.expand(3, 40))
    il.iris_fp8_mm(C, il.iris_fp8_empty(3, 0), B)
    assert torch.equal(C, torch.zeros_like(C))
    il.iris_fp8_mm(torch.empty((0, 40), dtype=torch.float32, device="cuda"), il.iris_fp8_empty(0, 256),
                   il.iris_fp8_empty(40, 256))
    il.iris_fp8_quantize(torch.empty((0, 7), dtype=torch.float16, device="cuda"), il.iris_fp8_empty(0, 7),
                         il.iris_fp8_empty(7, 0))
    e = torch.empty((0, 9), dtype=torch.float16, device="cuda")
    il.iris_fp8_swiglu(il.iris_fp8_empty(0, 9), e, e)
    torch.cuda.synchronize()


# ---------------------------------------------------------- gated activation

def check_computed(q, want, what):
    """8-bit values of computed numbers: half an e4m3 step off `want`, itself good to 1e-5."""
    codes, scales = parts(q)
    err = 1e-5
    amax = ref.block_amax(want, 1)
    lo, hi = ref.scale_bytes(amax * (1 - err)), ref.scale_bytes(amax * (1 + err))
    assert np.all((scales == lo) | (scales == hi)), f"{what}: scales"
    sc = ref.spread(scales, 1, codes.shape)
    got = ref.decode(codes) * sc
    a = np.abs(want) * (1 + err)
    step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(a / sc, 2.0 ** -30))) - 3), ref.SUB)
    off = ~(np.abs(got - want) <= 0.5 * step * sc + err * np.abs(want))
    assert not off.any(), (what, int(off.sum()), np.argwhere(off)[0].tolist(), got[off][0], want[off][0])
    assert_untouched(q, what)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_swiglu(rows, cols, dtype):
    note(f"swiglu {rows}x{cols} {dtype}")
    both, bv = on_gpu(sample(rows, 2 * cols, rows + cols), dtype)   # halves of one matrix
    gate, up, g, u = both[:, :cols], both[:, cols:], bv[:, :cols], bv[:, cols:]
    h, gk, uk = (fresh(rows, cols) for _ in range(3))
    il.iris_fp8_swiglu(h, gate, up, gk, uk)
    check_computed(h, ref.swiglu(g, u), "h")
    check_quantized(gk, g, 1, "gate")
    check_quantized(uk, u, 1, "up")
    h2 = fresh(rows, cols)
    il.iris_fp8_swiglu(h2, gate, up)
    for x, y in zip(parts(h), parts(h2)):
        assert np.array_equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_swiglu_extremes(dtype):
    """Large gates of both signs (sigmoid 0 and 1), NaN and infinities stay where they are."""
    g = np.tile(np.array([-1e4, -200.0, -100.0, -90.0, -20.0, -0.0, 0.0, 20.0, 90.0, 1e4, 1.0, 2.0]), (4, 11))
    u = sample(4, g.shape[1], 3)
    u[2] = 1.0
    gt, gv = on_gpu(g, dtype)
    ut, uv = on_gpu(u, dtype)
    h = fresh(4, g.shape[1])
    note(f"swiglu extremes {dtype}")
    il.iris_fp8_swiglu(h, gt, ut)
    check_computed(h, ref.swiglu(gv, uv), "h")
    ut[1, 5] = float("nan")
    gt[3, 8] = float("inf")
    il.iris_fp8_swiglu(h, gt, ut)
    nan = np.zeros(g.shape, bool)
    nan[1, 5] = nan[3, 8] = True
    assert np.array_equal((parts(h)[0] & 0x7f) == 0x7f, nan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_swiglu_bwd(rows, cols, dtype):
    note(f"swiglu_bwd {rows}x{cols} {dtype}")
    gk, uk = made(sample(rows, cols, 1)), made(sample(rows, cols, 2))
    g, u = ref.values(*parts(gk)), ref.values(*parts(uk))
    dh, dv = on_gpu(sample(rows, cols, 3) / 64, dtype, cols + 3, 1) if cols % 2 else on_gpu(sample(rows, cols, 3) / 64, dtype)
    out = [fresh(rows, cols), fresh(rows, cols)] + [fresh(cols, rows) for _ in range(3)]
    dg, du, dgt, dut, ht = out
    il.iris_fp8_swiglu_bwd(dg, du, dh, gk, uk, dgt, dut, ht)
    wg, wu = ref.swiglu_bwd(g, u, dv)
    e = 1e-5 * (1 + np.abs(g))      # differences of the formula in 64 bits
    ng = dv * (ref.swiglu(g + e, u) - ref.swiglu(g - e, u)) / (2 * e)
    assert np.all(np.abs(wg - ng) <= 1e-8 * (1 + np.abs(dv)) * (1 + np.abs(u)) * (1 + np.abs(g)))
    for q, want, what in ((dg, wg, "dgate"), (du, wu, "dup"), (dgt, wg.T, "dgate_t"), (dut, wu.T, "dup_t"),
                          (ht, ref.swiglu(g, u).T, "h_t")):
        check_gradient(q, want, wg_size(g, u, dv, what), what)
    alone = [fresh(rows, cols), fresh(rows, cols)]
    il.iris_fp8_swiglu_bwd(alone[0], alone[1], dh, gk, uk)
    one = fresh(cols, rows)
    il.iris_fp8_swiglu_bwd(alone[0], alone[1], dh, gk, uk, None, None, one)
    for x, y in ((alone[0], dg), (alone[1], du), (one, ht)):
        for s, t in zip(parts(x), parts(y)):
            assert np.array_equal(s, t)


def wg_size(g, u, dh, what):
    """What 1e-5 is relative to: dgate is a sum of s and g s (1 - s) that may cancel."""
    s = ref.sigmoid(g)
    if what == "dgate":
        return np.abs(dh * u) * s * (1 + np.abs(g) * (1 - s))
    if what == "dgate_t":
        return (np.abs(dh * u) * s * (1 + np.abs(g) * (1 - s))).T
    return None


def check_gradient(q, want, size, what):
    want = np.ascontiguousarray(want)
    size = np.abs(want) if size is None else np.ascontiguousarray(size)
    codes, scales = parts(q)
    err = 1e-5
    amax, slack = ref.block_amax(want, 1), err * ref.block_amax(size, 1)
    lo, hi = ref.scale_bytes(np.maximum(amax - slack, 0.0)), ref.scale_bytes(amax + slack)
    assert np.all((scales == lo) | (scales == hi)), f"{what}: scales"
    sc = ref.spread(scales, 1, codes.shape)
    got = ref.decode(codes) * sc
    a = np.abs(want) + err * size
    step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(a / sc, 2.0 ** -30))) - 3), ref.SUB)
    off = ~(np.abs(got - want) <= 0.5 * step * sc + err * size)
    assert not off.any(), (what, int(off.sum()), np.argwhere(off)[0].tolist(), got[off][0], want[off][0])
    assert_untouched(q, what)


def from_gpu(x):
    """An Fp8 operand of x's values, made by the library (whose codes other tests compare bit for bit)."""
    q = il.iris_fp8_empty(*x.shape)
    il.iris_fp8_quantize(torch.from_numpy(x).to(torch.float32).cuda(), q)
    return q


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2432, 2432), (2433, 2437)])
def test_swiglu_bwd_of_many_tiles(rows, cols, dtype):
    """More than 341 tiles: one workgroup forms all results of a tile, its second
    turn in the shared memory of the first. Every choice of the transposed outputs
    gives the same bits as all of them together."""
    note(f"swiglu_bwd {rows}x{cols} {dtype}")
    gk, uk = from_gpu(sample(rows, cols, 1)), from_gpu(sample(rows, cols, 2))
    g, u = ref.values(*parts(gk)), ref.values(*parts(uk))
    dh, dv = on_gpu(sample(rows, cols, 3) / 64, dtype, *((cols + 3, 1) if cols % 2 else ()))
    wg, wu = ref.swiglu_bwd(g, u, dv)
    wants = {"dgate": wg, "dup": wu, "dgate_t": wg.T, "dup_t": wu.T, "h_t": ref.swiglu(g, u).T}
    whole = None
    for turned in (("dgate_t", "dup_t", "h_t"), (), ("dgate_t",), ("dup_t",), ("h_t",), ("dgate_t", "dup_t"),
                   ("dgate_t", "h_t"), ("dup_t", "h_t")):
        note(f"  with {turned}")
        out = {k: fresh(rows, cols) for k in ("dgate", "dup")}
        out.update({k: fresh(cols, rows) for k in turned})
        il.iris_fp8_swiglu_bwd(out["dgate"], out["dup"], dh, gk, uk, out.get("dgate_t"), out.get("dup_t"), out.get("h_t"))
        if whole is None:
            whole = out
            for k, q in out.items():
                check_gradient(q, wants[k], wg_size(g, u, dv, k), k)
            again = {k: fresh(*q.shape) for k, q in out.items()}
            il.iris_fp8_swiglu_bwd(again["dgate"], again["dup"], dh, gk, uk, again["dgate_t"], again["dup_t"], again["h_t"])
            out = again
        for k, q in out.items():
            assert torch.equal(q.codes.view(torch.uint8), whole[k].codes.view(torch.uint8)), (turned, k)
            assert torch.equal(q.scales.view(torch.uint8), whole[k].scales.view(torch.uint8)), (turned, k)
            assert_untouched(q, k)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 200), (200, 300), (2432, 2433)])
def test_swiglu_bwd_nan_and_infinities_stay_where_they_are(rows, cols):
    """NaN and infinities in dh and NaN codes in the kept gate give NaN codes there, and all else is as if zeros stood there."""
    note(f"swiglu_bwd special values {rows}x{cols}")
    rng = np.random.default_rng(rows)
    at = np.zeros((rows, cols), bool)
    at[rng.integers(0, rows, 60), rng.integers(0, cols, 60)] = True
    kept = np.zeros((rows, cols), bool)
    kept[rng.integers(0, rows, 20), rng.integers(0, cols, 20)] = True
    base = sample(rows, cols, 3)
    specials = np.array([np.nan, np.inf, -np.inf])[rng.integers(0, 3, (rows, cols))]
    results = []
    for filled in (False, True):
        dh, _ = on_gpu(np.where(at, specials if filled else 0.0, np.where(kept, 0.0, base)), "bf16")
        gk, uk = from_gpu(np.where(at | kept, 0.0, sample(rows, cols, 1))), from_gpu(np.where(at | kept, 0.0, sample(rows, cols, 2)))
        if filled:
            gk.codes.view(torch.uint8)[torch.from_numpy(kept).cuda()] = 0x7f
        out = [fresh(rows, cols), fresh(rows, cols)] + [fresh(cols, rows) for _ in range(3)]
        il.iris_fp8_swiglu_bwd(out[0], out[1], dh, gk, uk, *out[2:])
        results.append([(c if i < 2 else c.T, s) for i, (c, s) in enumerate(parts(q) for q in out)])
    for i, ((want, ws), (got, gs)) in enumerate(zip(*results)):
        nan = kept if i == 4 else at | kept                 # h does not depend on dh
        assert np.array_equal(ws, gs), i
        assert np.array_equal((got & 0x7f) == 0x7f, nan), i
        assert np.array_equal(got[~nan], want[~nan]), i


# --------------------------------------------------------- streams and graphs

@pytest.mark.gpu
def test_other_stream_and_graph_replay():
    """All operators on a side stream, and captured: every replay gives what the eager calls gave."""
    M, H, K = 192, 384, 512
    x = torch.from_numpy(sample(M, K, 1)).to(torch.float16).cuda()
    wg, wd = made(sample(2 * H, K, 2, 0.0) / 20, 128), made(sample(K, H, 3, 0.0) / 20, 128)
    x8, h8 = il.iris_fp8_empty(M, K), il.iris_fp8_empty(M, H)
    gk, uk = il.iris_fp8_empty(M, H), il.iris_fp8_empty(M, H)
    gu = torch.empty((M, 2 * H), dtype=torch.float16, device="cuda")
    y = torch.empty((M, K), dtype=torch.float16, device="cuda")
    dg, du = il.iris_fp8_empty(M, H), il.iris_fp8_empty(M, H)
    dgt = il.iris_fp8_empty(H, M)
    dh = torch.from_numpy(sample(M, H, 4)).to(torch.float16).cuda()

    def step():
        il.iris_fp8_quantize(x, x8)
        il.iris_fp8_mm(gu, x8, wg)
        il.iris_fp8_swiglu(h8, gu[:, :H], gu[:, H:], gk, uk)
        il.iris_fp8_mm(y, h8, wd)
        il.iris_fp8_swiglu_bwd(dg, du, dh, gk, uk, dgt)

    def results():
        torch.cuda.synchronize()
        return [y.clone(), gu.clone()] + [torch.from_numpy(p) for q in (x8, h8, gk, uk, dg, du, dgt) for p in parts(q)]

    step()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    for a, b in zip(results(), want):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        y.fill_(7.0)
        gu.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        for a, b in zip(results(), want):
            assert torch.equal(a, b)
        step()
        for a, b in zip(results(), want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_split_products_of_threads_that_share_a_stream():
    """Split contractions from several host threads, on one stream (one workspace) and on streams of their own."""
    note("split products from threads")
    M, N, K = 260, 390, 4100
    assert il.iris_fp8_mm_workspace_size(M, N, K) > 0
    ops = [(made(sample(M, K, t)), made(sample(N, K, 10 + t, 0.0) / np.sqrt(K), 128)) for t in range(4)]
    wants = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in ops]
    for (A, B), C in zip(ops, wants):
        il.iris_fp8_mm(C, A, B)
    torch.cuda.synchronize()
    for streams in ([torch.cuda.current_stream()] * 4, [torch.cuda.Stream() for _ in ops]):
        outs = [[torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(30)] for _ in ops]
        torch.cuda.synchronize()

        def calls(t):
            for C in outs[t]:
                il.iris_fp8_mm(C, *ops[t], stream=streams[t])
        threads = [threading.Thread(target=calls, args=(t,)) for t in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for t in range(4):
            assert all(torch.equal(C, wants[t]) for C in outs[t]), t


@pytest.mark.gpu
def test_more_blocks_than_a_launch_holds():
    """2^29 blocks and more, at 8 threads a block, are more threads than one launch can have."""
    rows = (1 << 29) + 1000
    x = (torch.arange(rows, device="cuda", dtype=torch.int32) % 2039).to(torch.float16).reshape(rows, 1)
    q = il.Fp8(torch.zeros((rows, 16), dtype=torch.uint8, device="cuda")[:, :1],
               torch.zeros((rows, 1), dtype=torch.uint8, device="cuda"))

    def same_as_alone(call):
        for start in (0, (1 << 28) - 500, (1 << 29) - 500, rows - 1000):
            p = il.iris_fp8_empty(1000, 1)
            call(p, x[start:start + 1000])
            for big, small in ((q.codes, p.codes), (q.scales, p.scales.view(torch.uint8))):
                assert torch.equal(big[start:start + 1000], small.view(torch.uint8))
    note("quantize 2^29 blocks")
    il.iris_fp8_quantize(x, q)
    same_as_alone(lambda p, v: il.iris_fp8_quantize(v, p))
    note("swiglu 2^29 blocks")
    il.iris_fp8_swiglu(q, x, x)
    same_as_alone(lambda p, v: il.iris_fp8_swiglu(p, v, v))


@pytest.mark.gpu
def test_mm_of_more_small_tiles_than_a_launch_holds():
    """2^30 rows of A and one of B: 2^24 tiles of 64 x 64."""
    M, K = 1 << 30, 16
    note("mm 2^30 rows")
    codes = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")            # ones
    codes[:, 3] = torch.arange(M, device="cuda", dtype=torch.int32).remainder_(7).to(torch.uint8).mul_(8)   # 0, 2^-6 .. 2^-1
    scales = torch.full((M, 4), 127, dtype=torch.uint8, device="cuda")
    B = put(np.full((1, K), 0x38, np.uint8), np.full((1, 1), 127, np.uint8))
    C = torch.zeros((M, 1), dtype=torch.float16, device="cuda")
    il.iris_fp8_mm(C, il.Fp8(codes, scales[:, :1]), B)
    want = 15.0 + torch.tensor([0.0] + [2.0 ** -i for i in range(6, 0, -1)], dtype=torch.float16, device="cuda")
    for start in range(0, M, 1 << 28):
        at = torch.arange(start, start + (1 << 28), device="cuda", dtype=torch.int32).remainder_(7)
        assert torch.equal(C[start:start + (1 << 28), 0], want[at])


@pytest.mark.gpu
def test_split_products_in_graphs_on_streams_and_in_a_callers_workspace():
    """The library's workspace, its first use within a capture, on a stream of its own and on the current one; a
    caller's of just the size asked for, holding NaN."""
    M, N, K = 301, 397, 4111
    note("split products: workspaces")
    need = il.iris_fp8_mm_workspace_size(M, N, K)
    assert need > 0 and plan(M, N, K, "bf16")[2] > 1
    A, B = from_gpu(sample(M, K, 1)), made(sample(N, K, 2, 0.0) / np.sqrt(K), 128)
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    il.iris_finalize()                                  # no workspace is there
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        il.iris_fp8_mm(C, A, B)
    want = torch.empty_like(C)
    il.iris_fp8_mm(want, A, B)
    check_product(want, ref.values(*parts(A)), ref.values(*parts(B), 128), None, None, "bf16", "eager")
    for _ in range(3):
        C.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)
        il.iris_fp8_mm(C, A, B)                         # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(C, want)
    other = torch.cuda.Stream()
    C.fill_(7.0)
    torch.cuda.synchronize()
    il.iris_fp8_mm(C, A, B, stream=other)
    other.synchronize()
    assert torch.equal(C, want)
    ws = torch.full((need // 4 + 64,), float("nan"), dtype=torch.float32, device="cuda")
    for _ in range(2):
        C.fill_(7.0)
        il.iris_fp8_mm(C, A, B, workspace=ws[:need // 4])
        assert torch.equal(C, want) and bool(ws[need // 4:].isnan().all())
    with pytest.raises(il.IrisError, match="WORKSPACE"):
        il.iris_fp8_mm(C, A, B, workspace=ws[:need // 4 - 1])

@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(3, 40), (70, 90), (90, 300), (200, 130), (700, 1100), (2300, 2100)])
def test_mm_of_nothing_in_every_kernel(M, N):
    """K = 0: the bias and the old value alone, from the kernel for few rows and from tiles."""
    note(f"mm {M}x{N}x0")
    A, B = il.iris_fp8_empty(M, 0), il.iris_fp8_empty(N, 0, 128)
    bias = torch.arange(M, dtype=torch.float32, device="cuda")
    C = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    il.iris_fp8_mm(C, A, B)
    assert torch.equal(C, torch.zeros_like(C))
    along_m = dict(config=il.Config(flags=il.IRIS_FLAG_BIAS_ALONG_M))
    il.iris_fp8_mm(C, A, B, bias, **along_m)
    assert torch.equal(C, bias[:, None].expand(M, N))
    il.iris_fp8_mm(C, A, B, bias, accumulate=True, **along_m)
    assert torch.equal(C, 2 * bias[:, None].expand(M, N))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 1 << 21), (40, (1 << 21) - 77), (90, 1 << 21), (200, (1 << 21) - 77), (200, 1 << 21)])
def test_mm_of_the_longest_contraction(M, K):
    """2^21 products of -1, 0 and 1: every sum is exact, whatever its order."""
    N = 70
    note(f"mm {M}x{N}x{K}")
    rng = np.random.default_rng(M)
    a, b = (rng.integers(-1, 2, (n, K)).astype(np.int8) for n in (M, N))
    one = np.array([0xb8, 0x00, 0x38], np.uint8)
    A, B = put(one[a + 1], np.full((M, -(-K // 128)), 127, np.uint8)), put(one[b + 1], np.full((N, -(-K // 128)), 127, np.uint8))
    want = a.astype(np.float32) @ b.T.astype(np.float32)     # below 2^24
    for dtype in ("fp32", "fp16"):
        C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
        il.iris_fp8_mm(C, A, B)
        assert torch.equal(C.cpu(), torch.from_numpy(want).to(DT[dtype]))
