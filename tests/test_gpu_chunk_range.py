"""When the dense attention reports HS_ERR_RANGE, and when not: scores far below the others, queries
that nothing is computed with."""
import numpy as np
import pytest

import cache_plain as CP
from test_gpu_cache_ops import RANGE, Cache, check_chunk, make_q, run_chunk, torch

pytestmark = pytest.mark.gpu


def low_rows(rng, n, n_low):
    """n rows, the first n_low of which score -2.4e8 and less on the queries of low_q."""
    x = rng.standard_normal((n, 576)) / 32
    x[:, 0] = 0
    x[:n_low, 0] = 4096.0
    return CP.pack_rows(x[:, :512], x[:, 512:])


def low_q(rng, n, heads):
    q = make_q(rng, n, heads, "bf16")
    q[:, :, 0] = -60000.0
    return q


@pytest.mark.parametrize("n,n_low,tokens", [(200, 70, 1), (200, 128, 9), (4000, 3000, 1), (4000, 3990, 3), (3000, 2000, 40)])
@pytest.mark.parametrize("heads", [16, 64])
def test_rows_of_very_low_scores_before_others(heads, n, n_low, tokens):
    """Their weight is 0 by the formula, in whatever tile or part of the context they are: no error.
    A query that sees them alone has no score in range and is reported. With 40 segments the parts
    are joined row by row, with fewer by several threads' slices."""
    rng = np.random.default_rng(n + tokens)
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(-(-n // 64),)) as c:
        rows = low_rows(rng, n, n_low)
        c.put_rows(0, 0, np.arange(n), rows)
        q = low_q(rng, tokens, heads)
        segs = tokens if tokens == 40 else 1
        start = np.arange(tokens + 1) if segs > 1 else np.array([0, tokens])
        limit = n - np.arange(tokens) % 4
        out, lse = run_chunk(c, 0, [0] * segs, start, limit, q, 1.0)
        assert c.pool.get_error() == 0
        check_chunk(c, [CP.row_values(rows)[n_low:]], [0] * segs, start, limit - n_low, q, 1.0, out, lse, "bf16")
        limit[tokens // 2] = n_low
        out, lse = run_chunk(c, 0, [0] * segs, start, limit, q, 1.0)
        assert c.pool.get_error() == RANGE
        assert torch.all(out[tokens // 2] == 0) and torch.all(torch.isneginf(lse[tokens // 2]))
        check_chunk(c, [CP.row_values(rows)[n_low:]], [0] * segs, start, limit - n_low, q, 1.0, out, lse, "bf16",
                    set(range(tokens)) - {tokens // 2})


def test_scores_next_to_the_lower_border():
    """The largest scores at -2,879,488 in two later tiles, others at -2,940,928 before them: in range,
    and the largest share the weight. All scores at -3,084,288: none in range."""
    with Cache(heads=16, n_layers=1, lpi=1, pages=(4,)) as c:
        n, t = 200, np.arange(200)
        x = np.zeros((n, 576))
        x[:, 0], x[:, 1], x[:, 2] = t < 70, (t >= 70) & (t < 140), t >= 140
        rows = CP.pack_rows(x[:, :512], x[:, 512:])
        c.put_rows(0, 0, t, rows)
        q = torch.zeros(2, 16, 576, dtype=torch.float16, device="cuda")
        q[0, :, 0], q[0, :, 1], q[0, :, 2] = -45952.0, -44992.0, -44992.0
        q[1, :, :3] = -48192.0
        out, lse = run_chunk(c, 0, [0], [0, 2], [n, n], q, 64.0)
        assert c.pool.get_error() == RANGE
        assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
        first, _ = run_chunk(c, 0, [0], [0, 1], [n], q[:1], 64.0)
        assert c.pool.get_error() == 0 and torch.equal(first[0], out[0])
        wo, wl, _, _ = CP.attend(q[0].double().cpu().numpy(), CP.row_values(rows), 64.0)
        # equal weights, rounded to fp16 (2^-11); exact values; the output's 2^-11. Scores at 2^22 log2
        # units are held to 2^-2 of one, their reference as well
        assert np.all(np.abs(out[0].double().cpu().numpy() - wo) <= 1.01 * 2.0 ** -10 * np.abs(wo))
        assert np.all(np.abs(lse[0].cpu().numpy() - wl) <= 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads", [16, 64])
def test_queries_of_tokens_that_see_nothing(heads, dtype):
    """Padding tokens inside a segment (limit 0) may hold anything, NaN and infinities too: their
    output is 0 and nothing is reported, until one of them sees a row."""
    rng = np.random.default_rng(heads)
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(3,)) as c:
        x = rng.standard_normal((150, 576))
        rows = CP.pack_rows(x[:, :512], x[:, 512:])
        c.put_rows(0, 0, np.arange(150), rows)
        q = make_q(rng, 30, heads, "bf16").to(dtype)
        limit = 150 - np.arange(30)
        blind = [1, 8, 9, 10, 15, 29]
        limit[blind] = 0
        q[1], q[8, 3, 575], q[9, :, 0], q[10] = float("nan"), float("inf"), float("-inf"), float("nan")
        q[15, heads - 1, 64:128] = float("nan")
        q[29] = float("inf")
        name = "bf16" if dtype is torch.bfloat16 else "fp16"
        clean = q.clone()
        clean[blind] = 0
        for start in ([0, 30], [0, 9, 11, 30]):
            segs = len(start) - 1
            out, lse = run_chunk(c, 0, [0] * segs, start, limit, q, 1 / 24)
            assert c.pool.get_error() == 0
            check_chunk(c, [CP.row_values(rows)], [0] * segs, start, limit, clean, 1 / 24, out, lse, name)
        for j in blind:                                # one row seen: reported, and that query alone
            one = limit.copy()
            one[j] = 1
            out, lse = run_chunk(c, 0, [0], [0, 30], one, q, 1 / 24)
            assert c.pool.get_error() == RANGE, j
            check_chunk(c, [CP.row_values(rows)], [0], [0, 30], limit, clean, 1 / 24, out, lse, name, set(range(30)) - {j})
