"""e4m3 codes with a power-of-two scale for each block, and the layer built on them, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

"bitsandbytes deep dive", sections 5.1 (blockwise scales) and 8.1 - 8.3 (a storage format apart from the compute
dtype).  Readings taken: the OCP 8-bit float E4M3 (bias 7, largest value 448, no infinity, NaN 0x7F), blocks of
128 x 128 of a weight and of 1 x 128 of activations, the scale 2^(e - 127) with the least byte e that brings a block's
largest magnitude to 448 or less; codes to nearest, ties to even; a block that is not finite has e = 255 and codes 0.
"""
import numpy as np

from . import bf16, f16

FORMATS = {"bf16": bf16, "f16": f16}
BLOCK = 128
# the 127 values of codes 0 .. 126, ascending
VALUES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def decode(codes):
    """Values of e4m3 codes (uint8), float64."""
    codes = np.asarray(codes, dtype=np.uint8)
    v = np.append(VALUES, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -v, v)


def encode(z):
    """Codes of |z| <= 448, to nearest, ties to even.  The values are ascending with the code and 127 of them: the
    code is the number of midpoints below |z| (at or below it, where the code below is odd)."""
    mag = np.abs(z)
    mid = (VALUES[1:] + VALUES[:-1]) / 2
    lo, hi = np.searchsorted(mid, mag, side="left"), np.searchsorted(mid, mag, side="right")
    c = np.where(lo % 2 == 0, lo, hi)            # lo: midpoints strictly below; a tie goes to the even code
    return (c | np.where(np.signbit(z), 0x80, 0)).astype(np.uint8)


def blocks(rows, cols, block_rows):
    return -(-rows // block_rows), -(-cols // BLOCK)


def quantize(bits, dtype="bf16", block_rows=BLOCK):
    """(codes uint8 [rows, cols], e uint8 [row of blocks, block]) of 16-bit patterns [rows, cols]."""
    x = FORMATS[dtype].to_f64(bits)
    rows, cols = x.shape
    br, bc = blocks(rows, cols, block_rows)
    codes, e = np.zeros((rows, cols), np.uint8), np.zeros((br, bc), np.uint8)
    for j in range(bc):
        part = x[:, j * BLOCK:(j + 1) * BLOCK]
        for i in range(br):
            blk = part[i * block_rows:(i + 1) * block_rows]
            if not np.isfinite(blk).all():
                e[i, j] = 255
                continue
            a = np.abs(blk).max()
            b = 0
            if a > 0:
                b = max(0, int(np.floor(np.log2(a))) - 10 + 127)
                while a > 448.0 * 2.0 ** (b - 127):
                    b += 1
            e[i, j] = b
            codes[i * block_rows:i * block_rows + blk.shape[0], j * BLOCK:j * BLOCK + blk.shape[1]] = \
                encode(blk / 2.0 ** (b - 127))
    return codes, e


def stored_scale(e, rows, block_rows):
    """The scale bytes as they are stored: [row of blocks, block] of a weight, [block, row] of rows, the last dimension
    padded with zeros to a multiple of 4."""
    e = e if block_rows == BLOCK else e.T
    return np.pad(e, ((0, 0), (0, -e.shape[1] % 4)))


def values(codes, e, block_rows=BLOCK):
    """The float64 values that codes stand for (NaN in a block that is not finite)."""
    rows, cols = codes.shape
    s = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    s = np.repeat(np.repeat(s, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]
    return decode(codes) * s


def dequantize(codes, e, block_rows=BLOCK, dtype="bf16"):
    """16-bit patterns of the values (which are fp32 values), rounded once."""
    return FORMATS[dtype].from_f32_rne(values(codes, e, block_rows).astype(np.float32))


def linear_fwd(xv, wv, xdrop=None, A=None, B=None, s=0.0):
    """(y, t) in float64 without any rounding, for the values xv [M, K] and wv [N, K]."""
    y = xv @ wv.T
    if A is None:
        return y, None
    t = s * (xdrop @ A)
    return y + t @ B, t
