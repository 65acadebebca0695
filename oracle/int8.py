"""int8 codes with one scale per row, and the layer built on them, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

"bitsandbytes deep dive", section 4: absmax int8 (s = 127 / max|x|, q = round(s x)) and
the vector-wise form, one scale for each row of x and each output of W.  Readings taken:
the rounding is decided in exact arithmetic, ties toward zero; the stored scale is
fl32(max|x| / 127); a code stands for RNE_16(fl32(scale * code)) in the compute dtype; a
row of zeros has scale 0 and codes 0; a row with an infinity or a NaN has scale NaN and
codes 0.
"""
import numpy as np

from . import bf16, f16

FORMATS = {"bf16": bf16, "f16": f16}


def quantize(bits, dtype="bf16"):
    """(codes int8 [rows, cols], scale float32 [rows]) of 16-bit patterns [rows, cols]."""
    x = FORMATS[dtype].to_f64(bits)
    ok = np.isfinite(x).all(axis=1)
    x = np.where(ok[:, None], x, 0.0)
    mag = np.abs(x)
    a = mag.max(axis=1)
    d = np.where(a > 0, a, 1.0)[:, None]
    # code = #{j >= 0 : 127 |x| / a > j + 1/2}; 254 |x| and (2j + 1) a are exact in float64
    j = np.floor(127.0 * mag / d)
    q = j + (254.0 * mag > (2.0 * j + 1.0) * d)
    codes = np.where(x < 0, -q, q).astype(np.int8)
    scale = (a.astype(np.float32) / np.float32(127.0)).astype(np.float32)
    return codes, np.where(ok, scale, np.float32(np.nan)).astype(np.float32)


def dequantize(codes, scale, dtype="bf16"):
    """16-bit patterns the codes stand for: RNE_16(fl32(scale * code))."""
    with np.errstate(invalid="ignore"):
        p = (scale[:, None].astype(np.float32) * codes.astype(np.float32)).astype(np.float32)
    return FORMATS[dtype].from_f32_rne(p)


def linear_fwd(xf, codes_x, scale_x, codes_w, scale_w, A=None, B=None, s=0.0):
    """(y, t) in float64, without any rounding: the int8 product with its scales, plus s (x A) B."""
    y = (codes_x.astype(np.float64) @ codes_w.astype(np.float64).T) * scale_x.astype(np.float64)[:, None] \
        * scale_w.astype(np.float64)[None, :]
    if A is None:
        return y, None
    t = s * (xf @ A)
    return y + t @ B, t


def linear_bwd_dx(dy, w16, A=None, B=None, s=0.0):
    """(u, dx) in float64 for the 16-bit values w16 [N, K] of the weight."""
    dx = dy @ w16
    if A is None:
        return None, dx
    u = s * (dy @ B.T)
    return u, dx + u @ A.T
