"""The limit of chunk_bits.py on the CPU: it passes the documented precision and no bit less."""
import numpy as np
import pytest

import cache_plain as CP
import chunk_bits as B


def bits(x, p):
    """x rounded to p significant bits, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, p)), e - p)


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_the_limit_tells_11_bits_from_10(seed):
    x, q, sm = B.data(seed)
    rng = np.random.default_rng(seed)
    v = CP.row_values(CP.pack_rows(x[:, :512], x[:, 512:]))
    kv, v = v, v[:, :512]
    weights = []
    for j in range(q.shape[0]):                        # against any reference, not the largest alone
        z = sm * (q[j].astype(np.float64) @ kv.T)
        weights.append(np.exp(z - z.max(axis=1, keepdims=True)) * 2.0 ** rng.uniform(0, 1, (q.shape[1], 1)))

    def error(p_bits, v_bits, out_bits=11):
        rounded = bits(v, v_bits)
        want = np.array([p @ v / p.sum(axis=1, keepdims=True) for p in weights])
        got = np.array([bits(bits(p, p_bits) @ rounded / p.sum(axis=1, keepdims=True), out_bits) for p in weights])
        return B.relative_rms(got, want)
    assert error(11, 11) < 0.92 * B.LIMIT
    for p, w in ((10, 11), (11, 10), (8, 11), (11, 8)):
        assert error(p, w) > 1.1 * B.LIMIT, (p, w, error(p, w))
