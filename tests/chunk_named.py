"""Cached rows whose values name them, for the dense attention's tests: every score, weight and
value is a small integer or a power of two, so the formula's result is known to within the
output's rounding and a few sums, and a row, a page or a tile's scales taken wrongly show."""
import numpy as np

ONE = 0x38                       # the e4m3 code of 1
LN2 = float(np.float32(np.log(2.0)))
HEADS = [(0.0, 0.0), (1.0, 0.0), (0.0, 1.0), (1.0, -1.0)]     # (latent, rope) value of the queries of head h % 4


def exponents(n, kmax):
    """Exponent of the scales of each row's four groups [n, 4], 0 .. kmax, another one from row to
    row, from page to page and from group to group."""
    t, g = np.arange(n)[:, None], np.arange(4)[None, :]
    return (t * 5 + t // 64 + t // 256 + 3 * g) % (kmax + 1)


def rope_values(n):
    t = np.arange(n)
    return ((t * 3 + t // 64) % 7 - 3).astype(np.float64)


def rows(n, kmax):
    """[n, 656] bytes: row t has the code of 1 at dim t % 512, the scales 2^exponents and one rope
    value, and zeros elsewhere."""
    b = np.zeros((n, 656), np.uint8)
    t = np.arange(n)
    b[t, t % 512] = ONE
    b[:, 512:528] = np.ascontiguousarray(2.0 ** exponents(n, kmax), "<f4").view(np.uint8).reshape(n, 16)
    b[:, 528:530] = (rope_values(n).astype("<f4").view(np.uint32) >> 16).astype("<u2").view(np.uint8).reshape(n, 2)
    return b


def values(n, kmax):
    """The one value of each row that is not zero."""
    t = np.arange(n)
    return 2.0 ** exponents(n, kmax)[t, (t % 512) // 128]


def queries(n_tokens, heads):
    """[n_tokens, heads, 576] whose score of row t is a v_t + b r_t, (a, b) = HEADS[h % 4]."""
    q = np.zeros((n_tokens, heads, 576), np.float32)
    for h in range(heads):
        q[:, h, :512], q[:, h, 512] = HEADS[h % 4]
    return q


def attend(seen, n, kmax):
    """out [4, 512] and lse [4] of the four kinds of heads over the rows that `seen` [n] marks,
    with sm_scale = LN2, in 64 bits."""
    v, r, dim = values(n, kmax), rope_values(n), np.arange(n) % 512
    out, lse = np.zeros((4, 512)), np.full(4, -np.inf)
    if not seen.any():
        return out, lse
    for i, (a, b) in enumerate(HEADS):
        z = np.where(seen, LN2 * (a * v + b * r), -np.inf)
        w = np.exp(z - z.max())
        out[i] = np.bincount(dim, w * v, 512) / w.sum()
        lse[i] = z.max() + np.log(w.sum())
    return out, lse


# Bounds, n rows seen. The scores are integers from -3 to 11; times sm_scale log2 e, 1 to within
# 2^-23, they are off by less than 2^-19, and with exp2's 2^-22 a weight by less than 2^-18: in its
# fp16 form it is the power of two itself, in the sum it is as computed. A value is exact in fp16, and
# so are the sums of one dim: multiples of the smallest weight times value, fewer than 2^24 of them
# (2^16 between the smallest and the largest for n / 512 <= 10 rows of a dim; 2^11 for 79, 2^9 for 391).
# The weights' sum is off by 2^-24 for each of its additions: in a thread 16 for the first tile
# and one for each tile after, then the joins of threads and parts: fewer than n / 64 + 100. The
# quotient is rounded to the output type: half_step relative, 2^-25 at least.
def sums(n):
    return (n / 64 + 100) * 2.0 ** -24 + 2.0 ** -17


def out_bound(out, half_step, n):
    return np.maximum(half_step * np.abs(out), 2.0 ** -25) + 1.01 * sums(n) * np.abs(out)


def lse_bound(lse, n):
    return sums(n) + 2.0 ** -21 * (np.abs(lse) + 32)
