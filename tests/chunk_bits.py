"""How many bits the dense attention's weights and values have, from the size of its errors.

A number rounded to p significant bits is off by 2^(1 - p) / sqrt(12) of its binade's lower end,
root mean square: between 0.14 and 0.29 times 2^(1 - p) of itself, and 0.19 to 0.21 for mantissas
spread evenly in their logarithm. The values of different rows being independent of mean 0,
rounding the weights or the values leaves about that fraction of the output's own root mean
square, and so does rounding the output. With an fp16 output, and weights and values of 11 bits,
the three together are at most sqrt(3) 2^-10 0.21 = 3.6e-4 (3.1e-4 to 3.3e-4 when every step is
carried out on the data below); with 10 bits in one of them at least sqrt(4 + 2) 2^-10 0.165 =
3.9e-4 (4.2e-4 to 4.4e-4)."""
import numpy as np

LIMIT = 3.7e-4


def data(seed, n=900, tokens=8, heads=16):
    """Rows, queries (fp16) and sm_scale whose weights are spread over hundreds of rows, by an octave
    and more (a single heavy row would lend its own rounding to the whole output)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 576))
    q = (0.7 * rng.standard_normal((tokens, heads, 576))).astype(np.float16)
    return x, q, 1.0 / 24


def relative_rms(got, want):
    return float(np.sqrt(np.mean((got - want) ** 2) / np.mean(want ** 2)))
