"""The dropout oracle: known answers of the generator, the layout of its bits, and the mask's statistics."""
import numpy as np
import pytest

from oracle import dropout


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))])
def test_known_answers_of_ten_rounds(counter, key, want):
    """The published test vectors of the ten-round generator (zeros, ones, digits of pi)."""
    assert tuple(int(w) for w in dropout.philox4x32(counter, key, rounds=10)) == want


def test_rounds_by_hand():
    """Seven rounds against Python integers."""
    c, k = [7, 11, 0xDEADBEEF, 3], [0x12345678, 0x9ABCDEF0]
    got = [int(w) for w in dropout.philox4x32(tuple(c), tuple(k))]
    for _ in range(7):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b % 2 ** 32, (a >> 32) ^ c[3] ^ k[1], a % 2 ** 32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    assert got == c


def test_layout_and_independence_of_the_shape():
    seed, offset, p = (5 << 40) + 9, (1 << 35) + 77, 0.3
    m = dropout.mask(6, 100, p, seed, offset)
    w = dropout.philox4x32((3, 4, offset % 2 ** 32, offset >> 32), (seed % 2 ** 32, seed >> 32))
    for e in range(8):
        half = (int(w[e // 2]) >> (16 * (e % 2))) & 0xFFFF
        assert m[4, 24 + e] == (half >= dropout.threshold(p))
    assert np.array_equal(dropout.mask(3, 40, p, seed, offset), m[:3, :40])
    assert not np.array_equal(dropout.mask(6, 100, p, seed, offset + 1), m)
    assert not np.array_equal(dropout.mask(6, 100, p, seed + 1, offset), m)


@pytest.mark.parametrize("p", [0.0, 0.05, 0.5, 0.9, 65535 / 65536])
def test_rate_and_mean(p):
    n = 512 * 1024
    m = dropout.mask(512, 1024, p, 3, 4)
    q = dropout.threshold(p) / 65536
    # 6 standard deviations of a binomial count
    assert abs(int(m.sum()) - n * (1 - q)) <= 6 * np.sqrt(n * q * (1 - q)) + 1
    v = dropout.drop(np.ones((512, 1024)), p, 3, 4)
    assert set(np.unique(v)) <= {0.0, 65536 / (65536 - dropout.threshold(p))}


def test_dropped_values_are_zero_whatever_they_are():
    m = dropout.mask(4, 64, 0.5, 1, 2)
    x = np.where(m, 1.0, np.nan)
    assert np.array_equal(dropout.drop(x, 0.5, 1, 2), m * 2.0)
