"""Plain 64-bit forms of the 8-bit operators, for the tests alone (CPU, numpy).

The block scale and the e4m3 rounding are written from the format: a block's
scale is the smallest power of two (at least 2^-126) that brings its largest
finite magnitude to 448 or less; a code is sign, 4 exponent bits (bias 7), 3
mantissa bits, no infinity, largest value 448, smallest step 2^-9; rounding is
to nearest even.
"""
import numpy as np

BLK = 128
SUB = 2.0 ** -9      # e4m3 step below 2^-6
HALF = 2.0 ** -4     # half a step relative to the value's power of two
NAN_CODE = 0x7f


def decode_table():
    t = np.empty(256, np.float64)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = np.nan if (e == 15 and m == 7) else (-v if s else v)
    return t


TABLE = decode_table()


def decode(codes):
    return TABLE[np.asarray(codes, np.uint8)]


def encode(v):
    """float64 values (|v| <= 448 or not finite) -> codes, to nearest even."""
    v = np.asarray(v, np.float64)
    bad = ~np.isfinite(v)
    a = np.abs(np.where(bad, 0.0, v))
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    e = np.where(a >= np.exp2(e + 1), e + 1, np.where(a < np.exp2(e), np.maximum(e - 1, -6.0), e))
    q = np.rint(a / np.exp2(e - 3))      # mantissa in units of the step; rint rounds half to even
    e, q = np.where(q == 16, e + 1, e), np.where(q == 16, 8, q)
    code = np.where(q < 8, q, (e + 7) * 8 + (q - 8)).astype(np.uint8)
    return np.where(bad, NAN_CODE, code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def block_amax(x, block):
    """Largest finite magnitude of each block x 128 block."""
    rows, cols = x.shape
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    p = np.zeros((-(-rows // block) * block, -(-cols // BLK) * BLK))
    p[:rows, :cols] = a
    return p.reshape(p.shape[0] // block, block, -1, BLK).max(axis=(1, 3))


def scale_bytes(amax):
    """Smallest s >= 1 with amax / 2^(s-127) <= 448, found by trying."""
    s = np.ones(amax.shape, np.int64)
    for b in range(1, 255):
        s = np.where(amax * 2.0 ** (127 - b) > 448.0, b + 1, s)
    return np.where(amax == 0, 127, s).astype(np.uint8)


def spread(scales, block, shape):
    v = np.exp2(np.asarray(scales, np.float64) - 127.0)
    return v.repeat(block, 0)[:shape[0]].repeat(BLK, 1)[:, :shape[1]]


def quantize(x, block=1):
    """(codes, scale bytes) of float64 x (rows, cols)."""
    s = scale_bytes(block_amax(x, block))
    with np.errstate(invalid="ignore"):
        return encode(x / spread(s, block, x.shape)), s


def values(codes, scales, block=1):
    return decode(codes) * spread(scales, block, codes.shape)


def sigmoid(g):
    return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_bwd(g, u, dh):
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s
