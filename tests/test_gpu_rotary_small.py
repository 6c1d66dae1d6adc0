"""Rotations by angles next to the zeros of cosine and sine: each result relative to itself, in pairs of which one value is 0
so that nothing else covers it. Slow pairs at early positions, and steps next to whole quarters of a turn."""
import math
from fractions import Fraction

import numpy as np
import pytest

from test_gpu_cache_ops import Cache, i32, torch

pytestmark = pytest.mark.gpu

# The rest of the phase rounded to 24 bits (2^-24 of it, and of a cosine or sine of at most an eighth of a turn no more),
# sincospi within a unit in the last place (2^-23), the product with the value (2^-24); the other product is 0.
BOUND = 4 * 2.0 ** -24 * (1 + 2.0 ** -20)


@pytest.fixture(scope="module")
def pool():
    with Cache(heads=16, n_layers=1, lpi=1, pages=(2,)) as c:
        yield c.pool


def turned(phase):
    """Cosine and sine of a phase in 2^-64 turns, to the last bits of a double: of the rest behind the nearest quarter."""
    quarter = ((phase + (1 << 61)) >> 62) & 3
    rest = phase - (((phase + (1 << 61)) >> 62) << 62)
    w = float(Fraction(rest, 1 << 63)) * math.pi
    c, s = math.cos(w), math.sin(w)
    return ((c, s), (-s, c), (-c, -s), (s, -c))[quarter]


def wanted(pos, steps):
    out = np.empty((len(pos), len(steps), 2))
    for j, p in enumerate(np.asarray(pos).tolist()):
        for i, s in enumerate(steps.tolist()):
            out[j, i] = turned((p * s) % (1 << 64))
    return out


def rotate(pool, pos, steps, layout, a, b):
    """Pairs (a, b), each the same for a token, in 64-bit results [n, pairs, 2]."""
    n, k = len(pos), len(steps)
    x = torch.stack([a[:, None].expand(n, k), b[:, None].expand(n, k)], 2 if layout == "pairs" else 1).reshape(n, 2 * k).cuda()
    out = torch.full_like(x, 7.0)
    pool.rotary(i32(pos), steps.cuda(), [(x, out, layout)])
    g = out.double().cpu().numpy()
    return np.stack([g[:, 0::2], g[:, 1::2]] if layout == "pairs" else [g[:, :k], g[:, k:]], 2)


def check(pool, pos, steps, layout):
    rng = np.random.default_rng(len(pos))
    v, zero = torch.from_numpy(rng.uniform(0.5, 2.0, len(pos)).astype(np.float32)), torch.zeros(len(pos))
    w, x = wanted(pos, steps), v.double().numpy()[:, None]
    for a, b, want in ((v, zero, np.stack([x * w[:, :, 0], x * w[:, :, 1]], 2)), (zero, v, np.stack([-x * w[:, :, 1], x * w[:, :, 0]], 2))):
        got = rotate(pool, pos, steps, layout, a, b)
        err = np.abs(got - want)
        assert np.all(err <= BOUND * np.abs(want)), float((err / np.maximum(np.abs(want), 1e-300)).max())


@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("dims", [2, 6, 64, 256])
def test_early_positions_of_slow_pairs(pool, layout, dims):
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    f = [3.3e-6 * 0.7 ** i for i in range(dims // 2)]
    check(pool, [1, 2, 3, 5, 17, 100, 1023, -1, -2, -77], H.rotary_steps_of(f), layout)


def test_the_pairs_of_a_ramp(pool):
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    steps, _ = H.rotary_steps(64, 10000.0, "ramp", factor=40.0, original_ctx=4096.0)
    check(pool, list(range(1, 40)) + [4095, 131071, 1310719, -1], steps, "pairs")
    check(pool, list(range(1, 40)) + [4095, 131071, 1310719, -1], steps, "halves")


def test_angles_next_to_quarters_of_a_turn(pool):
    """A quarter and a little more or less, down to 2^-64 turns, of every quarter; and either side of the eighths, where
    the nearest quarter changes."""
    steps = []
    for e in (0, 3, 20, 31, 32, 33, 40, 55):
        steps += [(1 << 62) + (1 << e), (1 << 62) - (1 << e), (1 << 61) + (1 << e), (1 << 61) - (1 << e)]
    check(pool, [1, 2, 3, 4, 5, 6, 7, 8, -1, -2, -3, -5], torch.tensor(steps, dtype=torch.int64), "halves")
    check(pool, [1, 2, 3, 4, 5, 6, 7, 8, -1, -2, -3, -5], torch.tensor(steps, dtype=torch.int64), "pairs")


def test_a_single_step_of_a_phase(pool):
    """The least turn there is: 2^-64 of one, forwards and back."""
    check(pool, [1, -1, 2, 1 << 20, -(1 << 31)], torch.tensor([1] * 16, dtype=torch.int64), "pairs")
