"""The 4-bit weight format and its products in 64 bits, from their definition
(numpy and torch's roundings of single values only, no code of the library)."""
import numpy as np
import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def rounded(v, kind):
    """float32 values rounded to the type, as float64; beyond its range its
    largest value."""
    t = torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(TYPES[kind]).double().numpy()
    return np.where(np.isinf(t), np.copysign(torch.finfo(TYPES[kind]).max, t), t)


def nearest(w, s):
    """The whole number nearest to w / s for s > 0, ties to even.  (w has 24
    significant bits, s 11 and a whole or half number of up to 2^12 times s 24:
    the products and comparisons are exact in 64 bits.)"""
    t = np.clip(np.floor(w / s), -4096.0, 4096.0)
    t = np.where(t * s > w, t - 1, t)
    t = np.where((t + 1) * s <= w, t + 1, t)
    middle = (t + 0.5) * s
    return np.where((w > middle) | ((w == middle) & (t % 2 != 0)), t + 1, t)


def quantize(w, group, zeros, kind):
    """(codes N x K, scales and zero points N x groups) of an N x K matrix."""
    w = np.asarray(w, np.float64)
    N, K = w.shape
    ng = -(-K // group)
    codes, scales, points = np.zeros((N, K), np.uint8), np.zeros((N, ng)), np.zeros((N, ng), np.uint8)
    for j in range(ng):
        part = w[:, j * group:(j + 1) * group]
        bad = ~np.isfinite(part).all(axis=1)
        part = np.where(bad[:, None], 0.0, part)
        lo, hi = np.minimum(part.min(axis=1), 0), np.maximum(part.max(axis=1), 0)
        with np.errstate(over="ignore"):
            if zeros:
                s = (hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15)
            else:
                s = np.maximum(hi, -lo).astype(np.float32) / np.float32(7)
        s = rounded(s, kind)
        by = np.where(s > 0, s, 1.0)
        z = np.clip(nearest(-lo, by), 0, 15) if zeros else np.full(N, 8.0)
        z = np.where(s > 0, z, 0 if zeros else 8)
        q = np.clip(nearest(part, by[:, None]) + z[:, None], 0, 15)
        q = np.where(s[:, None] > 0, q, z[:, None])
        codes[:, j * group:(j + 1) * group] = np.where(bad[:, None], 0, q)
        scales[:, j] = np.where(bad, np.nan, s)
        points[:, j] = np.where(bad, 0, z)
    return codes, scales, points


def pack(codes):
    N, K = codes.shape
    c = np.zeros((N, -(-K // 32) * 32), np.uint8)
    c[:, :K] = codes
    return c[:, 0::2] | (c[:, 1::2] << 4)


def unpack(packed, K):
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(packed.shape[0], -1)[:, :K]


def values(codes, scales, points, group):
    """(values, s * (32 + q + z): the size of what a product's sums go through,
    which add (16 + q) x and take off (16 + z) x)."""
    K = codes.shape[1]
    s = np.repeat(scales, group, axis=1)[:, :K]
    z = np.repeat(points.astype(np.float64), group, axis=1)[:, :K]
    return s * (codes - z), np.abs(s) * (32 + codes + z)
