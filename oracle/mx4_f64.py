"""MXFP4 from its definition, in numpy and 64 bits: rows to codes and scales, and
the values that codes and scales stand for."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x, ceil=False):
    """x [M, K] (values of f32, bf16 or f16, in f64): codes uint8 [M, 16 G], two a
    byte, and scales uint8 [M, G]."""
    M, K = x.shape
    G = -(-K // 32)
    b = np.zeros((M, G * 32))
    b[:, :K] = x
    b = b.reshape(M, G, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    big = np.abs(b).max(axis=2)
    p = np.frexp(big)[1] - 1                  # big in [2^p, 2^(p+1))
    e = p - 2
    if ceil:
        e = np.where(big > 6.0 * np.ldexp(1.0, e), e + 1, e)
    e = np.where(big == 0, -127, np.maximum(e, -127))
    a = np.ldexp(np.abs(b), -e[:, :, None])
    code = np.zeros(a.shape, np.uint8)
    for lower in range(7):                    # past the point half way to the next value
        half = (GRID[lower] + GRID[lower + 1]) / 2
        code += ((a > half) | ((a == half) & (lower % 2 == 1))).astype(np.uint8)
    code += np.where(np.signbit(b), 8, 0).astype(np.uint8)
    code = np.where(bad[:, :, None], 0, code).astype(np.uint8).reshape(M, -1)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def values(codes, scales, K):
    """f64 [.., M, K]."""
    both = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1)
    v = GRID[both & 7] * np.where(both >= 8, -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        two = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
        return (v * np.repeat(two, 32, axis=-1))[..., :K]
