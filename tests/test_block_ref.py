"""The plain forms that the GPU tests of the block operators compare with: the generator
against its published known answers, gradients against differences."""
import numpy as np
import pytest

import block_ref as ref


def test_philox_known_answers():
    """The known answers that the generator's authors publish with it (philox 4x32, 10 rounds)."""
    f = 0xFFFFFFFF
    assert ref.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_mask_is_the_generators_halves():
    seed, offset, p = 0x123456789ABCDEF0, 0xFEDCBA9876543210, 0.3
    m = ref.mask(5, 21, p, seed, offset, row0=7)
    t = round(65536 * p)
    for i in range(5):
        for j in range(21):
            w = ref.philox([j // 8, i + 7, offset & 0xFFFFFFFF, offset >> 32], [seed & 0xFFFFFFFF, seed >> 32])[j % 8 // 2]
            u = w >> 16 if j % 2 else w & 0xFFFF
            assert m[i, j] == (65536 / (65536 - t) if u >= t else 0.0)


def test_mask_keeps_its_share():
    """A share of n independent values: within 5 standard deviations."""
    for p in (0.0, 0.1, 0.5):
        m = ref.mask(400, 500, p, 3, 4)
        q = round(65536 * p) / 65536
        assert abs((m == 0).mean() - q) <= 5 * np.sqrt(q * (1 - q) / m.size)


@pytest.mark.parametrize("kind", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slope_against_differences(kind):
    z = np.linspace(-8, 8, 801) + 0.003
    h = 1e-5   # the difference is off by h^2 / 6 of a third derivative below 10, and 2^-52 * 8 / h by cancelling
    d = (ref.act(z + h, kind) - ref.act(z - h, kind)) / (2 * h)
    assert np.max(np.abs(d - ref.slope(z, kind))) < 1e-9 + 2 ** -52 * 8 / h


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_norm_gradients_against_differences(layer, post):
    rng = np.random.default_rng(5)
    rows, cols, every = 5, 7, 2
    group = np.arange(rows) // every
    v = {"x": rng.normal(size=(rows, cols)), "y": rng.normal(size=(rows, cols)), "pre_w": rng.normal(size=cols),
         "pre_b": rng.normal(size=cols), "gate": rng.normal(size=(3, cols))}
    if post:
        v |= {"post_w": rng.normal(size=cols), "post_b": rng.normal(size=cols)}
    m = ref.mask(rows, cols, 0.3, 1, 2)
    dn, dr = rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols))

    def run(u):
        out, _ = ref.block_norm(u["x"], u["y"], layer=layer, pre_w=u["pre_w"], pre_b=u["pre_b"], post=post,
                                post_w=u.get("post_w"), post_b=u.get("post_b"), gate=u["gate"][group], alpha=0.7, m=m)
        return out

    out = run(v)
    got, _ = ref.block_norm_bwd(out["r"], out["stats"], dn, dr, v["y"], layer=layer, pre_w=v["pre_w"], post=post,
                                post_w=v.get("post_w"), post_b=v.get("post_b"), gate=v["gate"][group], alpha=0.7, m=m,
                                group=group)
    h = 1e-5
    for name, key in [("x", "dx"), ("y", "dy"), ("pre_w", "dpre_w"), ("pre_b", "dpre_b"), ("gate", "dgate")] + \
            ([("post_w", "dpost_w"), ("post_b", "dpost_b")] if post else []):
        for at in np.ndindex(v[name].shape):
            two = []
            for s in (h, -h):
                u = dict(v, **{name: v[name].copy()})
                u[name][at] += s
                o = run(u)
                two.append((o["n"] * dn).sum() + (o["r"] * dr).sum())
            d = (two[0] - two[1]) / (2 * h)
            assert abs(d - got[key][at]) < 1e-7 * max(1.0, np.abs(got[key]).max()), (name, at)
