"""Steps of rotary positions (host arithmetic, no GPU): the frequencies of every scaling as whole
2^-64 turns per position, and what is refused."""
import ctypes
import math
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

# pi to 60 digits, so that a turn is known far beyond 2^-64
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


@pytest.fixture(scope="module")
def H():
    from sparse_mla_kv_indexer_gb300 import build
    build.build()
    from sparse_mla_kv_indexer_gb300 import hisparse
    return hisparse


def turns_apart(step, frequency):
    """How far a step is from a frequency (a double, taken as exact), in turns, around the circle."""
    want = Fraction(frequency) / (2 * PI)
    d = (Fraction(int(step) % (1 << 64), 1 << 64) - want) % 1
    return float(min(d, 1 - d))


def formula(dims, theta, scaling, factor=1.0, original_ctx=0.0, beta_fast=32.0, beta_slow=1.0):
    half = range(dims // 2)
    if scaling == "theta":
        theta = theta * factor ** (dims / (dims - 2))
    f = [theta ** (-2 * i / dims) for i in half]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "ramp":
        at = lambda b: dims * math.log(original_ctx / (2 * math.pi * b)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), dims - 1)
        r = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in half]
        f = [x * (1 - t) + x / factor * t for x, t in zip(f, r)]
    return f


@pytest.mark.parametrize("dims", [2, 4, 64, 96, 256])
@pytest.mark.parametrize("scaling,more", [("none", {}), ("linear", {"factor": 8.0}), ("theta", {"factor": 4.0}),
                                          ("ramp", {"factor": 40.0, "original_ctx": 4096.0}),
                                          ("ramp", {"factor": 2.5, "original_ctx": 100.0, "beta_fast": 8.0, "beta_slow": 2.0})])
def test_steps_are_the_frequencies_in_turns(H, dims, scaling, more):
    if scaling == "theta" and dims == 2:
        with pytest.raises(H.HisparseError):
            H.rotary_steps(dims, 10000.0, scaling, **more)
        return
    steps, magnitude = H.rotary_steps(dims, 10000.0, scaling, **more)
    assert steps.shape == (dims // 2,) and magnitude == 1.0
    for s, f in zip(steps.tolist(), formula(dims, 10000.0, scaling, **more)):
        # a frequency of at most 1: a power, a few products and a quotient in double, each off by 2^-53 of
        # its value or (pow) a unit of 2^-52
        assert turns_apart(s, f) <= 2.0 ** -50, (s, f)


def test_own_frequencies_of_any_sign_and_size(H):
    f = [0.0, 1.0, -1.0, 1024.0, -1024.0, 2 * math.pi, 1e-300, -1e-300, math.pi, 3.5]
    for s, x in zip(H.rotary_steps_of(f).tolist(), f):
        assert turns_apart(s, x) <= 2.0 ** -53 * (abs(x) + 2), x


def test_the_magnitude_of_a_ramp(H):
    _, m = H.rotary_steps(64, 10000.0, "ramp", factor=40.0, original_ctx=4096.0, magnitude=0.1)
    assert abs(m - (1 + 0.1 * math.log(40.0))) <= 2.0 ** -24 * 1.5
    _, m = H.rotary_steps(64, 10000.0, "linear", factor=40.0, magnitude=0.1)
    assert m == 1.0


def test_refusals(H):
    bad = [dict(dims=0), dict(dims=3), dict(dims=-2), dict(dims=258), dict(theta=0.0), dict(theta=-1.0),
           dict(theta=float("nan")), dict(theta=float("inf")), dict(scaling="linear", factor=0.0),
           dict(scaling="linear", factor=float("nan")), dict(scaling="theta", factor=-2.0),
           dict(scaling="ramp", factor=4.0), dict(scaling="ramp", factor=4.0, original_ctx=4096.0, beta_fast=0.0),
           dict(scaling="ramp", factor=4.0, original_ctx=4096.0, beta_slow=float("nan")),
           dict(scaling="ramp", theta=1.0, factor=4.0, original_ctx=4096.0),
           dict(scaling="ramp", factor=4.0, original_ctx=4096.0, magnitude=float("inf")),
           dict(scaling="linear", factor=1e-4)]                      # frequencies beyond the largest
    for b in bad:
        with pytest.raises(H.HisparseError):
            H.rotary_steps(**{**dict(dims=64, theta=10000.0), **b})
    with pytest.raises(ValueError):
        H.rotary_steps(64, 10000.0, "other")
    for f in ([], [1025.0], [float("nan")], [float("inf")], [1.0] * 129):
        with pytest.raises(H.HisparseError):
            H.rotary_steps_of(f)
    one, m = (ctypes.c_uint64 * 1)(), ctypes.c_float(0.0)
    assert H.lib.hs_rotary_steps(None, one, ctypes.byref(m)) == 1
    assert H.lib.hs_rotary_steps_of(1, None, one) == 1
