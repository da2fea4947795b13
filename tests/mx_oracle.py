"""The microscaled formats and products in 64 bits, from their definition
(numpy only, no code of the library)."""
import numpy as np

BLOCK = 32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
GRID = {"e2m1": E2M1, "e4m3": E4M3}


def nearest(v, grid):
    """Index of the grid value nearest to |v|; at a midpoint the even one."""
    mid = (grid[1:] + grid[:-1]) / 2
    m = np.abs(v)
    low, high = np.searchsorted(mid, m, "left"), np.searchsorted(mid, m, "right")
    return np.where(low % 2 == 0, low, high)


def exponents(amax, fmt):
    """Scale exponents of blocks whose largest magnitudes are amax > 0."""
    frac, e = np.frexp(amax)  # amax = frac * 2^e, 0.5 <= frac < 1
    e = e.astype(np.int64)
    return e - 1 - 2 if fmt == "e2m1" else e - 1 - 8 + (frac * 2 > 1.75)


def quantize(x, fmt):
    """(element codes rows x blocks x 32, scale bytes rows x blocks)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = np.zeros((rows, nb * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, nb, BLOCK)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    amax = np.abs(v).max(axis=2) if nb else np.zeros((rows, 0))
    e = np.where(amax > 0, exponents(np.where(amax > 0, amax, 1.0), fmt), -127).clip(-127, 127)
    y = np.ldexp(v, -e[:, :, None])
    top = 8 if fmt == "e2m1" else 128
    codes = nearest(y, GRID[fmt]) + np.where(np.signbit(y), top, 0)
    codes = np.where(bad[:, :, None], 0, codes)
    return codes.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(codes, fmt):
    rows = codes.shape[0]
    c = codes.reshape(rows, -1)
    return c[:, 0::2] | (c[:, 1::2] << 4) if fmt == "e2m1" else c


def values(packed, scales, cols, fmt):
    """float64 values of a packed matrix."""
    rows, nb = scales.shape
    if fmt == "e2m1":
        c = np.stack([packed & 15, packed >> 4], axis=2).reshape(rows, nb, BLOCK)
        v = np.concatenate([E2M1, -E2M1])[c]
    else:
        half = np.concatenate([E4M3, [np.nan]])
        v = np.concatenate([half, -half])[packed.reshape(rows, nb, BLOCK)]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * s[:, :, None]).reshape(rows, nb * BLOCK)[:, :cols]


def round_trip(x, fmt):
    codes, scales = quantize(x, fmt)
    return values(pack(codes, fmt), scales, np.asarray(x).shape[1], fmt)
