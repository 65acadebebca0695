"""The dropout mask of the LoRA branch, in integer arithmetic.

TEST INFRASTRUCTURE ONLY (see the package docstring).

"bitsandbytes deep dive", section 12 (LoraConfig(..., lora_dropout=0.05)).  The page names no generator; taken:
Philox-4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011,
whose multipliers and key increments these are), key = seed, counter = (column // 8, row, offset), 16 bits for each of
8 columns, kept at or above round(65536 p).
"""
import numpy as np

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85
LOW = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key, rounds=7):
    """Four uint32 words for counters (four arrays or integers) under a key of two integers."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k0, k1 = key
    for _ in range(rounds):
        a, b = c[0] * np.uint64(M0), c[2] * np.uint64(M1)            # < 2^64: exact
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & LOW, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & LOW]
        k0, k1 = (k0 + W0) & 0xFFFFFFFF, (k1 + W1) & 0xFFFFFFFF
    return [v.astype(np.uint32) for v in c]


def threshold(p):
    return int(np.rint(np.float64(p) * 65536.0))


def mask(rows, cols, p, seed, offset):
    """Boolean [rows, cols]: what is kept."""
    groups = (cols + 7) // 8
    g, m = np.meshgrid(np.arange(groups), np.arange(rows))
    w = philox4x32((g, m, np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)),
                   (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([h for x in w for h in (x & 0xFFFF, x >> 16)], axis=2).reshape(rows, 8 * groups)[:, :cols]
    return bits >= threshold(p)


def drop(v, p, seed, offset):
    """drop(v) in float64: kept values over 1 - p, zero elsewhere (whatever is dropped)."""
    keep = mask(*v.shape, p, seed, offset)
    return np.where(keep, v, 0.0) * (65536.0 / (65536.0 - threshold(p)))
