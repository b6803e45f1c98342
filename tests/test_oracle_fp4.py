"""The 4-bit oracle, pinned independently of itself."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import fp4


def test_grid_from_the_bits():
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        v = Fraction(m, 2) if e == 0 else Fraction(2 + m, 2) * 2 ** (e - 1)
        assert fp4.e2m1_decode(c) == (-1 if c & 8 else 1) * v


def test_encode_worked_ties():
    # halfway between neighbours: to the even mantissa
    for v, mag in [(0.25, 0), (0.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (3.5, 4), (5.0, 4), (6.5, 6), (1e30, 6)]:
        for sign in (1, -1):
            c = fp4.e2m1_encode(np.float32(sign * v))
            assert fp4.e2m1_decode(c) == sign * mag and (c >> 3) == (sign < 0), v
    assert fp4.e2m1_encode(np.float32(-0.0)) == 8


def test_encode_is_nearest():
    v = np.concatenate([np.linspace(-8, 8, 4001), np.random.default_rng(0).standard_normal(2000) * 3])
    got = np.abs(fp4.e2m1_decode(fp4.e2m1_encode(v)) - v)
    best = np.abs(v[:, None] - np.concatenate([fp4.MAGNITUDES, -fp4.MAGNITUDES])).min(1)
    assert np.array_equal(got, best)


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantise_bounds(fmt):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 192)) * np.exp2(rng.integers(-40, 40, (40, 1)))).astype(np.float32)
    codes, sf, g = fp4.quantize(x, fmt)
    v = fp4.values(codes, sf, g, fmt)
    d = np.repeat(fp4.scale_bytes_to_values(sf, fmt), fp4.GROUP[fmt], axis=1) * (1 if g is None else g[:, None].astype(float))
    # half the widest step (1 between 4 and 6); E4M3 scales round by up to 1/16, subnormal ones by up to 2^-10
    # of the unit, so a value may pass 6 s g by that
    slack = 1.0 + (6 / 16 if fmt == 0 else 0)
    sub = 0 if fmt == 1 else 6 * 2.0 ** -10 * g[:, None].astype(float)
    assert np.all(np.abs(v - x) <= d * slack * (1 + 1e-6) + sub)
    if fmt == 1:
        amax = np.abs(x).reshape(40, -1, 32).max(2)
        s = fp4.scale_bytes_to_values(sf, 1)
        assert np.all(amax <= 6 * s) and np.all(amax > 3 * s)


def test_quantise_hand_worked():
    x = np.zeros((2, 64), np.float32)
    x[0, :4] = [6, -3, 1.25, 0.2]
    codes, sf, _ = fp4.quantize(x, 1)
    assert sf.tolist() == [[127, 0], [0, 0]]
    assert codes[0, :4].tolist() == [7, 0xD, 2, 0]
    x[0, 16] = 2688.0                       # rowmax: g = 1, the first group's s = E4M3(6 / 6) = 1
    codes, sf, g = fp4.quantize(x, 0)
    assert g[0] == 1.0 and g[1] == np.float32(2.0 ** -100)
    assert sf[0].tolist() == [0x38, 0x7E, 0, 0] and codes[0, :4].tolist() == [7, 0xD, 2, 0]
    assert codes[0, 16] == 7 and not codes[1].any()


def test_pack_and_blocked_layout():
    assert fp4.pack(np.array([[1, 2, 15, 0]])).tolist() == [[0x21, 0x0F]]
    c = np.random.default_rng(2).integers(0, 16, (3, 64)).astype(np.uint8)
    assert np.array_equal(fp4.unpack(fp4.pack(c)), c)
    sf = np.arange(1, 1 + 130 * 6, dtype=np.int64).reshape(130, 6) % 251 + 1
    out = fp4.tile_scales(sf.astype(np.uint8), 0).reshape(2, 2, 32, 4, 4)      # row tile, block, r % 32, r / 32, j % 4
    for r, j in [(0, 0), (31, 3), (32, 0), (127, 5), (128, 4), (129, 1)]:
        assert out[r // 128, j // 4, r % 32, r % 128 // 32, j % 4] == sf[r, j]
    assert not out[1, :, 2:].any() and not out[:, 1, :, :, 2:].any()


def test_planted_mistakes_are_seen():
    x = np.random.default_rng(3).standard_normal((4, 64)).astype(np.float32)
    codes, sf, g = fp4.quantize(x, 0)
    v = fp4.values(codes, sf, g, 0)
    assert not np.array_equal(fp4.values(codes, sf[:, ::-1], g, 0), v)                      # scales out of order
    assert not np.array_equal(fp4.values(fp4.unpack(fp4.pack(codes)[:, ::-1]), sf, g, 0), v)  # codes out of order
