"""The dense attention's documented precision: values of small scales, weights and values of 11
significant bits."""
import numpy as np
import pytest

import cache_plain as CP
import chunk_bits as B
from test_gpu_cache_ops import HALF_STEP, RANGE, Cache, check_chunk, make_q, run_chunk, torch

pytestmark = pytest.mark.gpu


def value_bound(kv, out, half_step):
    """Equal weights (sm_scale 0: every weight is the same power of two): a value is rounded once to
    fp16 after a product in fp32, at 4 times its size (2^-11 of it, 2^-27 at least, and 2^-24 of it);
    n sums in fp32; a quotient rounded to the output type (fp16: 2^-25 at least)."""
    v = np.abs(kv[:, :512])
    each = np.maximum(2.0 ** -11 * v, 2.0 ** -27) + 2.0 ** -24 * v
    return each.mean(0) + (v.shape[0] + 8) * 2.0 ** -23 * v.mean(0) + \
        np.maximum(half_step * 1.01 * np.abs(out), 2.0 ** -25)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("sizes", [(1e-2, 1e-3, 1e-4, 1e-6), (1.0, 1e-3, 1e-5, 1e-7), (1e-4, 3e-5, 1e-5, 1e-6),
                                   (3e-3, 7e-4, 1e-30, 16000.0)])
def test_values_of_small_scales(dtype, n, sizes):
    """Groups of normal and of tiny values, largest codes and small ones, in one row and in all rows."""
    rng = np.random.default_rng(n)
    with Cache(heads=16, n_layers=1, lpi=1, pages=(1,)) as c:
        x = rng.uniform(-1, 1, (n, 4, 128)) * np.array(sizes)[None, :, None]
        x[:, :, ::7] /= 60.0
        x[:, :, 5] = np.array(sizes)                   # a code of 448
        rows = CP.pack_rows(x.reshape(n, 512), rng.standard_normal((n, 64)))
        c.put_rows(0, 0, np.arange(n), rows)
        kv = CP.row_values(rows)
        q = make_q(rng, 2, 16, dtype)
        out, lse = run_chunk(c, 0, [0], [0, 2], [n, n], q, 0.0)
        assert c.pool.get_error() == 0
        want = kv[:, :512].mean(0)
        b = value_bound(kv, want, HALF_STEP[dtype])
        err = np.abs(out.double().cpu().numpy() - want)
        assert np.all(err <= b), ((err / b).max(axis=(0, 1)).reshape(4, 128).max(1), err.max())
        assert np.all(np.abs(lse.cpu().numpy() - np.log(n)) <= 2.0 ** -19)


@pytest.mark.parametrize("heads", [16, 64])
def test_a_cache_of_tiny_and_normal_groups(heads):
    """Rows whose groups differ by 10^7 in size, over several pages, within the bounds of any other."""
    rng = np.random.default_rng(heads)
    n = 700
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(11,)) as c:
        x = rng.standard_normal((n, 4, 128)) * np.array([1e-3, 1.0, 1e-5, 1e-4])[None, :, None]
        x[::3] *= 0.01
        rows = CP.pack_rows(x.reshape(n, 512), rng.standard_normal((n, 64)))
        c.put_rows(0, 0, np.arange(n), rows)
        kv = [CP.row_values(rows)]
        q = make_q(rng, 5, heads, "fp16")
        limit = np.arange(n - 4, n + 1)
        out, lse = run_chunk(c, 0, [0], [0, 5], limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, [0], [0, 5], limit, q, 1 / 24, out, lse, "fp16")
        # the groups of small values by themselves, with no absolute allowance but fp16's own steps
        for j in range(5):
            wo, _, a, s = CP.attend(q[j].double().cpu().numpy(), kv[0][:limit[j]], 1 / 24)
            b = 2.0 ** -11 * np.abs(wo) + (2 * CP.DZ * s[:, None] + 3 * 2.0 ** -11) * a + 2.0 ** -25 + 2.0 ** -27
            err = np.abs(out[j].double().cpu().numpy() - wo)
            assert np.all(err <= b), (j, (err / b).reshape(heads, 4, 128).max((0, 2)))


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("n", [900, 6000])
def test_weights_and_values_have_11_bits(heads, n):
    """The errors' root mean square, which a bit less in either would exceed (test_chunk_bits.py)."""
    x, q, sm = B.data(n, n=n, heads=heads)
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(-(-n // 64),)) as c:
        rows = CP.pack_rows(x[:, :512], x[:, 512:])
        c.put_rows(0, 0, np.arange(n), rows)
        kv = CP.row_values(rows)
        out, _ = run_chunk(c, 0, [0], [0, 8], [n] * 8, torch.from_numpy(q).cuda(), sm)
        assert c.pool.get_error() == 0
        want = np.array([CP.attend(q[j].astype(np.float64), kv, sm)[0] for j in range(8)])
        assert B.relative_rms(out.double().cpu().numpy(), want) < B.LIMIT


def test_small_rope_and_queries():
    """In fp16, rope and bf16 queries are exact from 2^-17 to 65504 and off by at most 2^-25 below; of one
    row seen, lse is the score: one exact product, then seven roundings to fp32 of numbers of its size (the
    scale, z, the reference, twice shifted, its sum with the logarithm and the factor of that): 2^-21 of it.
    Scores of 2,900,000 and more are out of range."""
    r = np.array([2.0 ** -e * m for e in (-15, -8, 0, 9, 14, 16, 17, 18, 20, 23, 25, 26, 40) for m in (1.0, 1.0078125, 1.9921875)])
    r = r[np.abs(r) <= 65504]
    with Cache(heads=16, n_layers=1, lpi=1, pages=(1,)) as c:
        for i, dtype in ((0, "bf16"), (0, "fp16"), (1, "bf16")):     # a small rope value, or a small query
            big = 49152.0
            for v in r:
                x = np.zeros((1, 576))
                x[0, 512] = v if i == 0 else big
                c.put_rows(0, 0, [0], CP.pack_rows(x[:, :512], x[:, 512:]))
                q = torch.zeros(1, 16, 576, dtype=torch.bfloat16 if dtype == "bf16" else torch.float16, device="cuda")
                q[..., 512] = big if i == 0 else float(v)
                out, lse = run_chunk(c, 0, [0], [0, 1], [1], q, 2.0 ** -10)
                z = v * big * 2.0 ** -10
                assert c.pool.get_error() == (RANGE if z > 2900000 else 0), (i, dtype, v)
                if z > 2900000:
                    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
                    continue
                off = 0 if v >= 2.0 ** -17 else 2.0 ** -25 * big * 2.0 ** -10
                assert np.all(np.abs(lse.double().cpu().numpy() - z) <= 1.01 * off + 2.0 ** -21 * abs(z) + 2.0 ** -19), (i, dtype, v)
