"""The division of the quantised append, enumerated on the CPU in whole numbers: with r the correctly
rounded 1 / s, q = x r and q + r (x - q s), each step rounded to fp32, is the correctly rounded
x / s for every amax / 448, and for x / scale next to every border between two codes."""
import numpy as np
import pytest


def round24(value, sticky):
    """value (whole numbers with four bits below a unit, any below those in sticky) rounded to 24
    significant bits, ties to even; in the same sixteenths."""
    w = 2 * value + sticky
    unit = np.where(value < 1 << 27, 16, np.where(value < 1 << 28, 32, 64)).astype(np.int64)
    low = w % unit
    down = w - low
    up = (low > unit // 2) | ((low == unit // 2) & (down // unit % 2 == 1))
    return (down + np.where(up, unit, 0)) // 2


def significant24(v):
    """Whole numbers below 2^31 rounded to 24 significant bits, ties to even."""
    a = np.abs(v)
    unit = np.ones_like(a)
    for k in range(24, 31):
        unit = np.where(a >= 1 << k, 1 << (k - 23), unit)
    low = a % unit
    a = a - low + np.where((low * 2 > unit) | ((low * 2 == unit) & (a // unit % 2 == 1)), unit, 0)
    return np.sign(v) * a


def kernel_quotient(x, s):
    """x / s as the kernel computes it, of 24-bit significands, in sixteenths of 2^-24 or, where
    x >= s, of 2^-23."""
    r = round24((1 << 51) // s, (1 << 51) % s != 0) // 16                 # 2^47 / s
    shift = np.where(x >= s, 24, 23)
    p = x * r                                                             # 2^47 x / s
    q = round24(p >> (shift - 4), p % (1 << (shift - 4)) != 0)
    d = (x << (51 - shift)) - q * s                                       # x - q s, in the same sixteenths of a unit
    t = significant24(d) * r                                              # times 2^47
    return round24(q + (t >> 47), (t & ((1 << 47) - 1)) != 0)


def true_quotient(x, s):
    n = x << np.where(x >= s, 27, 28)
    return round24(n // s, n % s != 0)


def test_every_amax_over_448():
    x = np.arange(1 << 23, 1 << 24, dtype=np.int64)
    s = np.full_like(x, 7 << 21)
    for a in range(0, x.size, 1 << 20):
        c = slice(a, a + (1 << 20))
        assert np.array_equal(kernel_quotient(x[c], s[c]), true_quotient(x[c], s[c]))


@pytest.mark.parametrize("seed", [None, 0, 1])
def test_quotients_next_to_the_borders_of_codes(seed):
    """Every x within 24 units of a border times the scale, for scales next to the multiples of 2^18
    (where such quotients come nearest to the middle between two fp32 numbers) and random ones."""
    if seed is None:
        s = (np.arange(32, 64, dtype=np.int64) << 18)[:, None] + np.arange(-24, 25)
        s = s[(s >= 1 << 23) & (s < 1 << 24)]
    else:
        s = np.random.default_rng(seed).integers(1 << 23, 1 << 24, 4000)
    border = np.arange(33, 64, 2, dtype=np.int64)                         # 5 significant bits and a half
    border = np.r_[border, border[::2] - 1]
    at = s[:, None] * border[None, :]                                     # 30 bits: 64 times the scale's
    x = (at >> 5)[:, :, None] + np.arange(-24, 25)                        # x / s = border / 32
    s = np.broadcast_to(s[:, None, None], x.shape)
    x = np.where(x >= 1 << 24, x >> 1, x)
    ok = (x >= 1 << 23) & (x < 1 << 24)
    x, s = x[ok], s[ok]
    assert x.size > 1_000_000 and np.array_equal(kernel_quotient(x, s), true_quotient(x, s))
