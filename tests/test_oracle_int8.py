"""The int8 oracle against exact rationals, the formulas against differences, and the rounding
argument of the GPU quantizer (one fma with a cut reciprocal decides every code) on the CPU."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import bf16, f16, int8

FMT = {"bf16": bf16, "f16": f16}


def _bits(fmt, v):
    return FMT[fmt].from_f32_rne(np.asarray(v, dtype=np.float32))


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_codes_match_rational_bruteforce(fmt):
    g = np.random.default_rng(5)
    rows = [g.standard_normal(64), g.standard_normal(64) * 1e-3, np.zeros(64), np.full(64, -3.0),
            np.arange(64) * 0.5, np.where(np.arange(64) == 7, 254.0, np.arange(64) + 0.0)]   # 254: x = (2j+1) are ties
    x = _bits(fmt, np.array(rows))
    codes, scale = int8.quantize(x, fmt)
    xf = FMT[fmt].to_f64(x)
    for i in range(x.shape[0]):
        a = max(Fraction(abs(v)) for v in xf[i])
        assert scale[i] == np.float32(np.float32(float(a)) / np.float32(127))
        for k in range(x.shape[1]):
            v = Fraction(xf[i, k])
            if a == 0:
                assert codes[i, k] == 0
                continue
            best = min(range(-127, 128), key=lambda j: (abs(127 * v / a - j), abs(j)))
            assert codes[i, k] == best
    assert codes[5, 1] == 0 and codes[5, 3] == 1 and codes[5, 7] == 127      # 0.5 -> 0, 1.5 -> 1: toward zero


def test_rows_that_are_not_finite():
    x = _bits("bf16", [[1.0, np.inf] * 32, [np.nan, 2.0] * 32, [1.0, -2.0] * 32])
    codes, scale = int8.quantize(x)
    assert np.isnan(scale[:2]).all() and not codes[:2].any()
    assert scale[2] == np.float32(2.0) / np.float32(127.0) and codes[2, 1] == -127 and codes[2, 0] == 63


def _fma_codes(x, a, fmt):
    """The GPU's decision in numpy: round(x * inv + 1.5 * 2^23) to fp32 with one rounding (the float64 sum of an
    exact 24 x 11-bit product and the constant is exact: 35 bits below 2^24), low byte."""
    pre = np.where((fmt == "bf16") & (a < 2.0 ** -100), np.float32(2.0 ** 100), np.float32(1.0)).astype(np.float32)
    inv = (np.float32(127.0) / (a * pre).astype(np.float32)).astype(np.float32) * np.float32(1.0 - 2.0 ** -21)
    s = (x * pre).astype(np.float64) * inv.astype(np.float32).astype(np.float64) + 12582912.0
    return (s.astype(np.float32).view(np.uint32) & 0xFF).astype(np.uint8).view(np.int8)


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_one_fma_decides_every_code(fmt):
    """Every mantissa of a against every magnitude up to it that can lie near a half-integer, and whole rows of
    random patterns over the format's exponents (subnormals, the largest values)."""
    m = FMT[fmt]
    mant = 128 if fmt == "bf16" else 1024
    one = 0x3F80 if fmt == "bf16" else 0x4C00                     # 1.0; 16.0 leaves fp16 room below
    g = np.random.default_rng(11)
    abits = (one + (np.arange(mant) if fmt == "bf16" else g.choice(mant, 96, replace=False))).astype(np.uint16)
    for ab in abits:
        lo = 0x3A00 if fmt == "bf16" else 0x2000
        xb = np.arange(lo, int(ab) + 1, dtype=np.uint16)
        row = np.concatenate([xb, xb | 0x8000]).astype(np.uint16)[None, :]
        want, _ = int8.quantize(row, fmt)
        got = _fma_codes(m.to_f32(row), m.to_f32(row[:, :1] * 0 + ab), fmt)
        assert np.array_equal(got, want), hex(int(ab))
    top = 0x7F7F if fmt == "bf16" else 0x7BFF
    for ab in [1, 2, 3, 0x7F, 0x80, 0x100, 0x0D00, top] + list(g.integers(1, top, 60)):
        xb = np.concatenate([g.integers(0, ab + 1, 4096), g.integers(max(0, ab - 2000), ab + 1, 4096), [ab]])
        row = (xb.astype(np.uint16) | (g.integers(0, 2, xb.size).astype(np.uint16) << 15))[None, :].astype(np.uint16)
        want, _ = int8.quantize(row, fmt)
        got = _fma_codes(m.to_f32(row), m.to_f32(row[:, :1] * 0 + np.uint16(ab)), fmt)
        assert np.array_equal(got, want), ab


def test_formulas_against_differences():
    """The layer is linear in x once the codes stand for values: differences of y along x are dx, and dA and dB
    are the differences of <dy, y> along A and B."""
    g = np.random.default_rng(7)
    M, N, K, r, s = 5, 6, 64, 3, 0.7
    w16 = bf16.to_f64(int8.dequantize(*int8.quantize(_bits("bf16", g.standard_normal((N, K))))))
    x16 = bf16.to_f64(int8.dequantize(*int8.quantize(_bits("bf16", g.standard_normal((M, K))))))
    A, B, dy = g.standard_normal((K, r)), g.standard_normal((r, N)), g.standard_normal((M, N))
    f = lambda x, A, B: float((dy * (x @ w16.T + s * (x @ A) @ B)).sum())
    u, dx = int8.linear_bwd_dx(dy, w16, A, B, s)
    grads = {"dx": dx, "dA": x16.T @ u, "dB": (s * (x16 @ A)).T @ dy}
    e = 1e-3
    for name, arr in (("dx", x16), ("dA", A), ("dB", B)):
        for _ in range(6):
            i = tuple(g.integers(0, d) for d in arr.shape)
            p, q = arr.copy(), arr.copy()
            p[i] += e
            q[i] -= e
            args = {"dx": lambda v: f(v, A, B), "dA": lambda v: f(x16, v, B), "dB": lambda v: f(x16, A, v)}[name]
            d = (args(p) - args(q)) / (2 * e)
            assert abs(d - grads[name][i]) <= 1e-9 * (1 + abs(d)) * 100
