"""The inputs and bounds of chunk_named.py themselves, on the CPU: the rows hold what the formulas
say, and a lost row, a lost page or the scales of another tile exceed the bounds."""
import numpy as np
import pytest

import cache_plain as CP
import chunk_named as N

HALF_STEP = 2.0 ** -11           # fp16


@pytest.mark.parametrize("kmax", [1, 3])
def test_the_rows_hold_the_formulas_values(kmax):
    n = 1500
    kv = CP.row_values(N.rows(n, kmax))
    t = np.arange(n)
    want = np.zeros((n, 576))
    want[t, t % 512] = N.values(n, kmax)
    want[:, 512] = N.rope_values(n)
    assert np.array_equal(kv, want)
    out, lse = N.attend(t < 1400, n, kmax)
    q = N.queries(1, 4)[0].astype(np.float64)
    wo, wl, _, _ = CP.attend(q, kv[:1400], N.LN2)
    assert np.allclose(out, wo, rtol=1e-12, atol=1e-15) and np.allclose(lse, wl, rtol=1e-12)


def lost(n, kmax, gone):
    """Whether the bounds tell the result without the rows `gone` from the whole."""
    all_rows = np.ones(n, bool)
    out, lse = N.attend(all_rows, n, kmax)
    all_rows[gone] = False
    less, _ = N.attend(all_rows, n, kmax)
    return bool((np.abs(out - less) > 2 * N.out_bound(out, HALF_STEP, n)).any())


@pytest.mark.parametrize("n,kmax", [(65, 3), (300, 3), (900, 3), (5000, 3), (40000, 2), (200003, 1)])
def test_the_bounds_see_a_lost_row_and_a_lost_page(n, kmax):
    rng = np.random.default_rng(n)
    for t in [0, 63, 64, n - 1, *rng.integers(0, n, 20)]:
        assert lost(n, kmax, [int(t)]), t
        assert lost(n, kmax, slice(int(t) // 64 * 64, int(t) // 64 * 64 + 64)) or n <= 64


@pytest.mark.parametrize("n,kmax", [(300, 3), (5000, 3), (200003, 1)])
def test_the_bounds_see_the_scales_of_another_tile(n, kmax):
    """The scales of the tile four before in one tile's place (the place they had in a ring of four)."""
    out, _ = N.attend(np.ones(n, bool), n, kmax)
    v, dim = N.values(n, kmax), np.arange(n) % 512
    e = N.exponents(n, kmax)
    for page in {4, max(4, n // 128), (n - 1) // 64}:
        t = np.arange(64 * page, min(64 * page + 64, n))
        w = v.copy()
        w[t] = 2.0 ** e[t - 256, (t % 512) // 128]
        stale = np.bincount(dim, w, 512) / n           # the head whose weights are all alike
        assert (np.abs(stale - out[0]) > 2 * N.out_bound(out[0], HALF_STEP, n)).any(), page
