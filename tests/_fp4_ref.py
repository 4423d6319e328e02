"""The cache in 4 bits of ``domino_verify.h`` in NumPy: its numbers, its bytes and the rounding, from the
definition, one candidate number at a time.  No code of the package is imported."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def powers(x):
    """Exponents of the blocks of 32 of x [..., d], 128 for blocks that are not finite."""
    x = np.asarray(x, np.float64)
    blocks = np.abs(x.reshape(x.shape[:-1] + (-1, 32)))
    with np.errstate(invalid="ignore"):
        top = blocks.max(-1)
    e = np.full(top.shape, -125)
    for i in range(-125, 125):
        e = np.where(top > 7 * 2.0 ** i, i + 1, e)
    return np.where(np.isfinite(blocks).all(-1), e, 128)


def codes(x, e):
    """Indices of the numbers of x's elements, sign bit 8 included; 0 in blocks that are not finite."""
    x = np.asarray(x, np.float64)
    y = x.reshape(x.shape[:-1] + (-1, 32)) / 2.0 ** e[..., None]
    with np.errstate(invalid="ignore"):
        far = np.abs(np.minimum(np.abs(y), 6.0)[..., None] - GRID)
    best = np.nan_to_num(far).min(-1, keepdims=True)
    # among the nearest the even index
    pick = np.where(far == best, np.where(np.arange(8) % 2 == 0, 2, 1), 0).argmax(-1)
    out = np.where(e[..., None] == 128, 0, pick + 8 * np.signbit(y))
    return out.reshape(x.shape).astype(np.uint8)


def values(code, e):
    """What codes [..., d] with exponents [..., d / 32] stand for."""
    x = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    with np.errstate(invalid="ignore"):
        two = np.where(e == 128, np.nan, 2.0 ** np.minimum(e, 127).astype(np.float64))
    return (x.reshape(x.shape[:-1] + (-1, 32)) * two[..., None]).reshape(x.shape)


def stored(x):
    """The numbers that stand for x in the cache."""
    e = powers(x)
    return values(codes(x, e), e)


def row_bytes(x):
    """Element bytes [..., d / 2] and power bytes [..., d / 32] of rows x [..., d]."""
    e = powers(x)
    c = codes(x, e)
    return c[..., 0::2] | (c[..., 1::2] << 4), (e + 127).astype(np.uint8)


def row_values(data, power):
    """The numbers of rows given by their bytes."""
    c = np.stack([data & 15, data >> 4], -1).reshape(data.shape[:-1] + (-1,))
    return values(c, power.astype(np.int64) - 127)
