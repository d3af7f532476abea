"""MXFP4 by its definition, in NumPy float64: codes, scales and the values they stand for."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = np.concatenate([GRID, -GRID])


def encode(v):
    """(codes [rows, KB, 32], scale bytes [rows, KB]) of the rows of a float64
    matrix: X the smallest integer with amax <= 6 2^X, codes by distance, ties
    to the even code; a block with a value that is not finite is all NaN."""
    rows, cols = v.shape
    kb = -(-cols // 32)
    p = np.zeros((rows, kb * 32))
    p[:, :cols] = v
    p = p.reshape(rows, kb, 32)
    bad = ~np.isfinite(p).all(-1)
    q = np.where(bad[..., None], 0.0, p)
    amax = np.abs(q).max(-1)
    X = np.full(amax.shape, -127)
    for x in range(-127, 128):                       # by trial: the first X that is large enough
        X = np.where((6.0 * 2.0 ** (x - 1) < amax) & (x > -127), x, X)
    y = q / np.ldexp(1.0, X)[..., None]
    d = np.abs(np.abs(y)[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    cand = d == best
    even = cand & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), np.argmax(even, -1), np.argmax(cand, -1))
    code = np.where(np.signbit(y), code + 8, code)
    code[bad] = 0
    return code.astype(np.uint8), np.where(bad, 255, X + 127).astype(np.uint8)


def pack(code):
    """[rows, KB, 32] codes -> [rows, KB*16] bytes, even element in the low half."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(code.shape[0], -1).astype(np.uint8)


def decode(packed, scales, cols):
    """float64 values [rows, cols] of packed codes and scale bytes."""
    code = np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1, 32)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    with np.errstate(invalid="ignore"):
        return (TABLE[code] * s[..., None]).reshape(packed.shape[0], -1)[:, :cols]


def decode_mxfp8(codes, scales):
    """float64 values of E4M3FN codes [rows, K] and scale bytes [rows, K/32]."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, np.ldexp(m / 8.0, -6), np.ldexp(1 + m / 8.0, e - 7))
    v = np.where((c & 127) == 127, np.nan, v)
    v = np.where(c >> 7, -v, v).reshape(codes.shape[0], -1, 32)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * s[..., None]).reshape(codes.shape[0], -1)
