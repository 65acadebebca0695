"""The fp8 oracle against brute force: nearest codes by distance over all of them, least scale by search, exact
rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

from bit_nf4_quantized_15_amd import workloads
from oracle import bf16, f16, fp8

FMT = {"bf16": (bf16, workloads.normal_bf16), "f16": (f16, workloads.normal_f16)}


def value(c):
    """E4M3 by its fields."""
    e, m = (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return None
    v = Fraction(m, 8) * Fraction(1, 64) if e == 0 else (1 + Fraction(m, 8)) * Fraction(2) ** (e - 7)
    return -v if c >> 7 else v


def test_values():
    got = fp8.decode(np.arange(256, dtype=np.uint8))
    for c in range(256):
        assert np.isnan(got[c]) if value(c) is None else Fraction(got[c]) == value(c)
    assert fp8.VALUES[-1] == 448.0


def nearest(z):
    """The code of an exact z by distance; ties to the even code."""
    best = min((abs(value(c) - abs(z)), c % 2, c) for c in range(127))
    return best[2]


def test_codes_are_the_nearest():
    g = np.random.default_rng(1)
    z = np.concatenate([fp8.VALUES, (fp8.VALUES[1:] + fp8.VALUES[:-1]) / 2, g.uniform(0, 448, 200),
                        2.0 ** g.uniform(-14, 8, 200), [2.0 ** -10, np.nextafter(2.0 ** -10, 1)]])
    for v, c in zip(z, fp8.encode(z)):
        assert c == nearest(Fraction(v)), v
    assert np.array_equal(fp8.encode(-z), fp8.encode(z) | 0x80)


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols,block_rows", [(3, 320, 1), (130, 192, 128), (1, 64, 128)])
def test_blocks(fmt, rows, cols, block_rows):
    m, normal = FMT[fmt]
    b = normal(rows + cols, (rows, cols), 1.0)
    b[0, :70] = 0
    x = m.to_f64(b)
    codes, e = fp8.quantize(b, fmt, block_rows)
    for i in range(e.shape[0]):
        for j in range(e.shape[1]):
            rs, cs = slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128)
            a = Fraction(np.abs(x[rs, cs]).max())
            least = next(k for k in range(256) if a <= 448 * Fraction(2) ** (k - 127))
            assert e[i, j] == least
            for v, c in list(zip(x[rs, cs].ravel(), codes[rs, cs].ravel()))[::7]:
                assert (c & 0x7F) == nearest(abs(Fraction(v)) / Fraction(2) ** (least - 127))
                assert bool(c >> 7) == bool(np.signbit(v))
    # half a step of e4m3 at most: 2^-4 of the value, or half the smallest subnormal of the block
    s = 2.0 ** (e.astype(float) - 127)
    full = np.repeat(np.repeat(s, block_rows, 0)[:rows], 128, 1)[:, :cols]
    assert (np.abs(fp8.values(codes, e, block_rows) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, full * 2.0 ** -10)).all()


def test_blocks_that_are_not_finite_and_stored_bytes():
    b = workloads.normal_bf16(3, (6, 256), 1.0)
    b[2, 5], b[4, 200] = 0x7F80, 0x7FC1
    codes, e = fp8.quantize(b, "bf16", 1)
    assert e[2, 0] == 255 and e[4, 1] == 255 and (e == 255).sum() == 2
    assert not codes[2, :128].any() and np.isnan(fp8.values(codes, e, 1)[2, :128]).all()
    assert fp8.stored_scale(e, 6, 1).shape == (2, 8) and not fp8.stored_scale(e, 6, 1)[:, 6:].any()
    assert fp8.stored_scale(np.ones((3, 5), np.uint8), 300, 128).shape == (3, 8)


def test_extreme_values():
    b = np.array([[0x0001] * 64, [0x7F7F] * 64, [0x0000] * 64, [0x8000] * 64], np.uint16)
    codes, e = fp8.quantize(b, "bf16", 1)
    assert e[0, 0] == 0 and codes[0, 0] == fp8.encode(np.array([2.0 ** -133 * 2.0 ** 127]))[0]
    assert e[1, 0] == 127 + 120 and e[2, 0] == 0 and codes[3, 0] == 0x80
