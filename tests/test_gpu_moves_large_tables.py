"""Moves in the tables of many requests of long contexts, where most entries name pages that stay: every entry of every
table, and every byte of the pages."""
import numpy as np
import pytest

from test_gpu_cache_ops import Cache, i32
from test_gpu_pages import Model, moved, spare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 7, 64, 65, 500])
@pytest.mark.parametrize("requests,max_ctx", [(96, 1 << 18), (301, 64 * 131)])
def test_moves_of_pages_that_many_tables_name(n, requests, max_ctx):
    """Tables full of random entries, placeholders among them, so that a moved page is named many times or never; there
    and back."""
    with Cache(n_layers=1, lpi=1, pages=(600,) + (1,) * (requests - 1), spare=n, max_ctx=max_ctx if max_ctx >= 600 * 64 else 600 * 64) as c:
        m = Model(c, requests)
        rng = np.random.default_rng(n)
        width = c.max_ctx // 64
        free, idx_free = spare(c)
        used, idx_used = ([p for p in range(c.n_pages) if p not in f] for f in (free, idx_free))
        for r in range(requests):
            bt, ix = rng.choice(used, width), rng.choice(idx_used, width)
            bt[rng.random(width) < 0.3] = -1
            m.set_pages(r, 0, bt=bt.tolist(), ix=ix.tolist())
        src, idx_src = rng.permutation(used)[:n], rng.permutation(idx_used)[:n]
        dst, idx_dst = np.array(free)[:n], np.array(idx_free)[:n]
        for a, b, ia, ib in ((src, dst, idx_src, idx_dst), (dst, src, idx_dst, idx_src)):
            c.pool.copy_pages(i32(a), i32(b), i32(ia), i32(ib), remap=True)
            moved(m, "kv", a, b, True)
            moved(m, "idx", ia, ib, True)
            assert c.pool.get_error() == 0
            m.check()
