"""4-bit codes with block scales: the codec, the quantiser, the blocked scale
layout and the value of the GEMM, written from the definitions.

TEST INFRASTRUCTURE ONLY (see the package docstring).

E2M1 has one sign, two exponent (bias 1) and one mantissa bit: magnitudes 0,
0.5, 1, 1.5, 2, 3, 4, 6.  Rounding is to nearest, ties to the even mantissa,
saturating; the sign is kept, also for results that round to zero.

Format 0 (E4M3 scale per 16, float32 per row), every step one float32
operation:  g = max(rowmax / 2688, 2^-100), s = E4M3(amax / (6 g)),
code = E2M1(x * (1 / (s g))), zero codes where s = 0.
Format 1 (UE8M0 scale per 32): s = 2^k, the smallest with amax <= 6 s,
k >= -127; code = E2M1(x / s) (exact quotient).
"""
from __future__ import annotations

import numpy as np

from .e4m3 import e4m3_decode, e4m3_encode

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GROUP = {0: 16, 1: 32}
_HALF = (MAGNITUDES[:-1] + MAGNITUDES[1:]) / 2


def e2m1_encode(v) -> np.ndarray:
    """Code (0..15) of each value: the index of the nearest magnitude; a value
    half way between two goes to the one of even index (mantissa bit 0)."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    below = (a[..., None] > _HALF).sum(-1)          # magnitudes that lie entirely below a
    tie = (a[..., None] == _HALF).any(-1)
    idx = np.where(tie & (below % 2 == 1), below + 1, below)
    return (idx | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def e2m1_decode(c) -> np.ndarray:
    c = np.asarray(c, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def pack(codes) -> np.ndarray:
    """[..., K] codes to [..., K/2] bytes, the even column in the low four bits."""
    c = np.asarray(codes, dtype=np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(q) -> np.ndarray:
    q = np.asarray(q, dtype=np.uint8)
    return np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)


def blocks(K: int, fmt: int) -> int:
    return -(-(K // GROUP[fmt]) // 4)


def tile_scales(sf, fmt: int) -> np.ndarray:
    """[M, J] scale bytes to the blocked layout; rows up to a multiple of 128
    and groups up to a multiple of four are zero.  Byte by byte."""
    M, J = sf.shape
    nb = -(-J // 4)
    out = np.zeros(-(-M // 128) * nb * 512, np.uint8)
    r, j = np.meshgrid(np.arange(M), np.arange(J), indexing="ij")
    out[((r // 128) * nb + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4] = sf
    return out


def scale_bytes_to_values(sf, fmt: int) -> np.ndarray:
    return e4m3_decode(sf) if fmt == 0 else np.exp2(np.asarray(sf, np.float64) - 127)


def quantize(x, fmt: int):
    """x [M, K] float32 (BF16 values): (codes [M, K], scale bytes [M, J], g [M] or None)."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    v = x.reshape(M, K // GROUP[fmt], GROUP[fmt])
    amax = np.abs(v).max(axis=2, initial=0).astype(np.float32)
    f = np.float32
    if fmt == 0:
        g = np.maximum(amax.max(axis=1, initial=0) / f(2688), f(2.0 ** -100)).astype(f)
        sf = e4m3_encode((amax / (g * f(6))[:, None]).astype(f))
        d = (e4m3_decode(sf).astype(f) * g[:, None]).astype(f)
        with np.errstate(divide="ignore"):
            r = np.where(d > 0, f(1) / d, f(0)).astype(f)
        y = (v * r[:, :, None]).astype(f)
    else:
        g = None
        # smallest k with amax <= 6 * 2^k, from a logarithm corrected by exact comparisons
        a = amax.astype(np.float64)
        k = np.floor(np.log2(np.where(a > 0, a / 6, 2.0 ** -127))).astype(np.int64)
        k = np.where(6 * np.exp2(k.astype(np.float64)) < a, k + 1, k)
        k = np.where(6 * np.exp2(k.astype(np.float64) - 1) >= a, k - 1, k)
        k = np.maximum(np.where(a > 0, k, -127), -127)
        sf = (k + 127).astype(np.uint8)
        y = v.astype(np.float64) / np.exp2(k.astype(np.float64))[:, :, None]
    return e2m1_encode(y).reshape(M, K), sf, g


def values(codes, sf, g, fmt: int) -> np.ndarray:
    """float64 values of codes [M, K]: exact products but for g."""
    v = e2m1_decode(codes) * np.repeat(scale_bytes_to_values(sf, fmt), GROUP[fmt], axis=1)
    return v if g is None else v * np.asarray(g, np.float64)[:, None]


def gemm(a, b):
    """Y = A B^T and T = sum |terms| of float64 values [M, K], [N, K]."""
    return a @ b.T, np.abs(a) @ np.abs(b).T
