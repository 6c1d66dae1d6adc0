"""Steps of rotary positions to the last of their 64 bits, and so the angle of every position whatever the frequency
(host arithmetic, no GPU)."""
import random
from fractions import Fraction

import pytest

from test_rotary_steps import PI, H  # noqa: F401

TURN = 1 << 64


def frequencies():
    rng = random.Random(7)
    some = [0.5, 1.0, 6.5, 12.5, 100.0, 999.9, 1000.0, 1023.999, 1024.0, 6.283185307179586, 3.141592653589793, 0.1, 1e-3, 3.3e-6,
            1e-12, 2.0 ** -64, 1e-18, 5e-324, 0.0]
    some += [rng.uniform(0, 1024) for _ in range(2000)] + [2.0 ** rng.uniform(-70, 10) for _ in range(2000)]
    # whole numbers of turns and what lies next to them in double
    some += [k * 6.283185307179586 for k in range(1, 163)] + [k * 6.283185307179586 * (1 - 2.0 ** -53) for k in range(1, 163)]
    return some + [-f for f in some]


def off(count, frequency, position=1):
    """How far `count` 2^-64 turns are from position x frequency (a double, taken as exact), in turns, around the circle."""
    d = (Fraction(count % TURN, TURN) - Fraction(frequency) * position / (2 * PI)) % 1
    return min(d, 1 - d)


def test_a_step_is_the_nearest_whole_number(H):  # noqa: F811
    f = frequencies()
    # rounded to the nearest: half of 2^-64; the arithmetic before it adds 2^-97 at most (a sum of 2^18 units of 2^-64 in
    # double; pi is known to 2^-190)
    most = Fraction(1, 1 << 65) * (1 + Fraction(1, 1 << 30))
    for at in range(0, len(f), 128):
        part = f[at:at + 128]
        for step, x in zip(H.rotary_steps_of(part).tolist(), part):
            assert off(step, x) <= most, x


@pytest.mark.parametrize("position", [1, 7, 1 << 20, (1 << 21) - 1, 1310719, (1 << 31) - 1, -(1 << 31), -1])
def test_the_angle_of_every_position(H, position):  # noqa: F811
    """What the header promises: within 2^-34 turns (2^31 times half a step; 1 + 2^-30 as above)."""
    f = frequencies()[::7]
    for at in range(0, len(f), 128):
        part = f[at:at + 128]
        for step, x in zip(H.rotary_steps_of(part).tolist(), part):
            assert off(step * position, x, position) <= Fraction(1, 1 << 34) * (1 + Fraction(1, 1 << 30)), (x, position)


def test_a_frequency_and_its_negative_turn_alike(H):  # noqa: F811
    f = [x for x in frequencies() if x > 0][:128]
    for a, b in zip(H.rotary_steps_of(f).tolist(), H.rotary_steps_of([-x for x in f]).tolist()):
        assert (a + b) % TURN == 0
