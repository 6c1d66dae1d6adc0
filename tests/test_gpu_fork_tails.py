"""Forks of one call whose tail pages are pages that other forks of the call copy rows from: which of the two came first
would decide what is copied, so the fork that would write there is not made, and the other ones are."""
import pytest

from test_gpu_cache_ops import BAD_ID, Cache, i32
from test_gpu_pages import Model, spare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("kind", ["kv", "idx"])
@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_a_tail_that_another_fork_copies_from(fmt, kind, order):
    with Cache(pages=(4, 3, 1, 1), fmt=fmt, spare=4) as c:
        m = Model(c, 4)
        t, ix = spare(c)
        tails, idx_tails = [t[0], t[1]], [ix[0], ix[1]]
        if kind == "kv":
            tails[0] = int(c.table[1][1])              # the page that the second fork copies six rows of
        else:
            idx_tails[0] = int(c.idx_table[1][1])
        args = [[0, 1], [2, 3], [70, 70], tails, idx_tails]
        c.pool.fork_requests(*[i32([a[k] for k in order]) for a in args])
        assert c.pool.get_error() == BAD_ID
        m.fork(1, 3, 70, tails[1], idx_tails[1])
        m.check()


def test_each_tail_the_other_forks_source():
    """Two that would swap their last pages: neither is made; a third one is."""
    with Cache(pages=(2, 2, 3, 1, 1, 1), spare=2) as c:
        m = Model(c, 6)
        t, ix = spare(c)
        c.pool.fork_requests(i32([0, 1, 2]), i32([3, 4, 5]), i32([65, 127, 150]),
                             i32([int(c.table[1][1]), int(c.table[0][1]), t[0]]),
                             i32([int(c.idx_table[1][1]), int(c.idx_table[0][1]), ix[0]]))
        assert c.pool.get_error() == BAD_ID
        m.fork(2, 5, 150, t[0], ix[0])
        m.check()


def test_tails_that_nothing_is_copied_from():
    """The same pages where they are not read: index tails that are not given, a last page that is whole, a source that is
    a placeholder read from the host, and the sources of forks that cannot be made."""
    with Cache(pages=(4, 3, 1, 1), spare=4) as c:
        m = Model(c, 4)
        t, ix = spare(c)
        last = int(c.table[1][1])
        m.set_pages(1, 1, bt=[-1], hp=[3])             # the page is the caller's again
        c.pool.fork_requests(i32([0, 1]), i32([2, 3]), i32([70, 70]), i32([last, t[0]]), i32([ix[0], ix[1]]))
        assert c.pool.get_error() == 0
        m.fork(0, 2, 70, last, ix[0])
        m.fork(1, 3, 70, t[0], ix[1])
        m.check()
        # an index page that is copied from is no tail of a call without index tails
        c.pool.fork_requests(i32([0, 1]), i32([2, 3]), i32([70, 70]), i32([t[1], t[2]]))
        assert c.pool.get_error() == 0
        m.fork(0, 2, 70, t[1], None)
        m.fork(1, 3, 70, t[2], None)
        m.check()
        # request 1's page 1 as a tail, where the other fork takes whole pages alone; sources and lengths out of range
        m.set_pages(1, 1, bt=[last])
        c.pool.fork_requests(i32([0, 1]), i32([2, 3]), i32([70, 64]), i32([last, t[0]]), i32([ix[0], ix[1]]))
        assert c.pool.get_error() == 0
        m.fork(0, 2, 70, last, ix[0])
        m.fork(1, 3, 64, t[0], ix[1])
        m.check()
        c.pool.fork_requests(i32([0, 4]), i32([2, 3]), i32([70, 70]), i32(t[:2]), i32(ix[:2]))
        assert c.pool.get_error() == BAD_ID
        m.fork(0, 2, 70, t[0], ix[0])
        c.pool.fork_requests(i32([0, 1]), i32([2, 3]), i32([70, c.max_ctx + 1]), i32(t[:2]), i32(ix[:2]))
        assert c.pool.get_error() == BAD_ID
        m.fork(0, 2, 70, t[0], ix[0])
        m.check()


def test_many_forks_of_which_some_write_where_others_read():
    """More forks than one CTA has threads: every fifth one's tail is the last page of another's source."""
    n = 300
    with Cache(pages=(2,) * n + (1,) * n, n_layers=1, lpi=1, spare=n) as c:
        m = Model(c, 2 * n)
        t, ix = spare(c)
        tails, idx_tails = t[:n], ix[:n]
        for k in range(0, n, 5):
            tails[k] = int(c.table[(k * 7 + 11) % n][1])
        src, length = list(range(n)), [65 + k % 63 for k in range(n)]
        length[11] = 64                                 # read by nobody: the first one's tail is free
        c.pool.fork_requests(i32(src), i32(range(n, 2 * n)), i32(length), i32(tails), i32(idx_tails))
        assert c.pool.get_error() == BAD_ID
        for k in range(n):
            if k % 5 or k == 0:
                m.fork(k, n + k, length[k], tails[k], idx_tails[k])
        m.check()
