"""The dense attention over rows that name themselves (chunk_named.py): every head's output and
lse within a few roundings of the formula, so that no row, page, cut of the work or tile's scales
can be taken wrongly unseen."""
import numpy as np
import pytest

import chunk_named as N
from test_gpu_cache_ops import HALF_STEP, Cache, dt, run_chunk, torch

pytestmark = pytest.mark.gpu


def check(out, lse, limit, n, kmax, dtype, tokens=None):
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    t = np.arange(n)
    for j in range(o.shape[0]) if tokens is None else tokens:
        wo, wl = N.attend(t < limit[j], n, kmax)
        for h in range(o.shape[1]):
            b = N.out_bound(wo[h % 4], HALF_STEP[dtype], limit[j])
            err = np.abs(o[j, h] - wo[h % 4])
            assert np.all(err <= b), (j, h, int(limit[j]), int((err / b).argmax()), float((err / b).max()))
            assert abs(l[j, h] - wl[h % 4]) <= N.lse_bound(wl[h % 4], limit[j]), (j, h, l[j, h], wl[h % 4])


def run(c, q, limit, start=None):
    start = [0, q.shape[0]] if start is None else start
    out, lse = run_chunk(c, 0, [0] * (len(start) - 1), start, limit, q, N.LN2)
    assert c.pool.get_error() == 0
    return out, lse


def queries(n, heads, dtype):
    return torch.from_numpy(N.queries(n, heads)).to(dt(dtype)).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("n", [1, 64, 65, 300, 900, 5000])
def test_a_few_tokens(n, heads, dtype):
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(-(-n // 64),)) as c:
        c.put_rows(0, 0, np.arange(n), N.rows(n, 3))
        limit = np.maximum(0, [n, n - 1, n // 2, n, max(1, n - 64)])
        limit[3] = 1
        out, lse = run(c, queries(5, heads, dtype), limit)
        check(out, lse, limit, n, 3, dtype, [j for j in range(5) if limit[j] > 0])


@pytest.mark.parametrize("heads,n", [(16, 700), (64, 333)])
def test_a_prompt_and_single_tokens_beside_it(heads, n):
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(-(-n // 64),)) as c:
        c.put_rows(0, 0, np.arange(n), N.rows(n, 3))
        rng = np.random.default_rng(n)
        limit = np.r_[np.arange(1, n + 1), rng.integers(1, n + 1, 90)]
        start = np.r_[0, n + np.arange(91)]
        out, lse = run(c, queries(n + 90, heads, "fp16"), limit, start)
        check(out, lse, limit, n, 3, "fp16", [*range(0, n, 17), *range(n, n + 90)])


@pytest.mark.parametrize("heads,n,kmax", [(16, 40000, 2), (64, 200003, 1)])
def test_long_contexts(heads, n, kmax):
    """One token, whose range is cut among all pairs, and two chunks."""
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(-(-n // 64),)) as c:
        c.put_rows(0, 0, np.arange(n), N.rows(n, kmax))
        out, lse = run(c, queries(1, heads, "fp16"), [n])
        check(out, lse, [n], n, kmax, "fp16")
        limit = np.r_[np.arange(n - 12, n + 1), [n // 2, n // 3, 77, n]]
        q = queries(17, heads, "fp16")
        out, lse = run(c, q, limit, [0, 9, 17])
        check(out, lse, limit, n, kmax, "fp16", [0, 5, 8, 9, 12, 13, 14, 15, 16])
        again, lse2 = run(c, q, limit, [0, 9, 17])
        assert torch.equal(out, again) and torch.equal(lse, lse2)
