"""The plain 64-bit forms of the 8-bit operators against torch's e4m3 type, by
brute force, and the gradient's formula against differences."""
import numpy as np
import torch

import fp8_ref as ref


def test_decode_matches_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.TABLE, equal_nan=True)


def test_encode_is_nearest_even_by_search():
    rng = np.random.default_rng(1)
    pos = ref.TABLE[:127]                       # 0 .. 448 ascending
    mid = (pos[1:] + pos[:-1]) / 2
    v = np.concatenate([pos, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng.uniform(0, 448, 20000),
                        np.exp2(rng.uniform(-14, 8.8, 20000))])
    got = ref.encode(v)
    d = np.abs(v[:, None] - pos[None])
    best = d.min(axis=1)
    even = [np.flatnonzero(row == b) for row, b in zip(d, best)]
    want = np.array([c[0] if len(c) == 1 or c[0] % 2 == 0 else c[1] for c in even], np.uint8)
    assert np.array_equal(got, want)
    assert np.array_equal(ref.encode(-v[1:]), want[1:] | 0x80)
    assert np.array_equal(ref.encode([np.nan, np.inf, -np.inf]), [0x7f] * 3)


def test_scale_is_the_smallest_power():
    a = np.array([[448.0, np.nextafter(448.0, 1e9), 449.0, 224.0, 225.0, 0.0, 1.0, 1.75, 1.7500001, 2.0 ** -133,
                   3.0e38]])
    s = ref.scale_bytes(a)[0]
    assert list(s[:9]) == [127, 128, 128, 126, 127, 127, 119, 119, 120]
    assert s[9] == 1 and 3.0e38 / 2.0 ** (int(s[10]) - 127) <= 448


def test_gradient_formula_against_differences():
    rng = np.random.default_rng(2)
    g, u, dh = rng.normal(size=(3, 500)) * 3
    e = 1e-5
    dg, du = ref.swiglu_bwd(g, u, dh)
    ng = dh * (ref.swiglu(g + e, u) - ref.swiglu(g - e, u)) / (2 * e)
    nu = dh * (ref.swiglu(g, u + e) - ref.swiglu(g, u - e)) / (2 * e)
    # a central difference is off by e^2 / 6 times a third derivative (below 1 for silu) plus rounding 2^-53 / e
    bound = (e * e + 1e-10) * (1 + np.abs(dh)) * (1 + np.abs(u)) * (1 + np.abs(g))
    assert np.all(np.abs(dg - ng) <= bound) and np.all(np.abs(du - nu) <= bound)
