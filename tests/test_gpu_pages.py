"""Forks of requests, copies and moves of pages and the tables read back, on the GPU against plain numpy
bookkeeping: tables and every byte of the pool."""
import numpy as np
import pytest

from test_gpu_cache_ops import BAD_ID, HOST_MISSING, INVALID, Cache, i32, torch

pytestmark = pytest.mark.gpu


class Model:
    """A pool of random bytes and what its tables and pages hold, kept in numpy."""

    def __init__(self, c, requests):
        self.c = c
        rng = np.random.default_rng(1)
        for t in c.kv + c.idx:
            t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
        c.host.copy_(torch.from_numpy(rng.integers(0, 256, tuple(c.host.shape), dtype=np.uint8)))
        n = c.max_ctx // 64
        self.bt, self.ix = np.full((requests, n), -1, np.int32), np.full((requests, n), -1, np.int32)
        self.hp = np.full((requests, n), -1, np.int64)
        for r, (a, b) in enumerate(zip(c.table, c.idx_table)):
            self.bt[r, :len(a)], self.ix[r, :len(b)] = a, b
        self.kv = [t.cpu().numpy().reshape(c.n_pages, 64, 656).copy() for t in c.kv]
        self.idx = [t.cpu().numpy().copy() for t in c.idx]

    def set_pages(self, r, first, bt=None, ix=None, hp=None):
        self.c.pool.set_pages(r, first, block_table=bt, idx_pages=ix, host_pages=hp)
        for t, v in ((self.bt, bt), (self.ix, ix), (self.hp, hp)):
            if v is not None:
                t[r, first:first + len(v)] = v

    def fork(self, src, dst, n, tail, idx_tail):
        k, rows = n // 64, n % 64
        for t in (self.bt, self.ix, self.hp):
            t[dst, :k] = t[src, :k]
        if not rows:
            return
        for layer, pages in enumerate(self.kv):
            p = self.bt[src, k]
            pages[tail][:rows] = (pages[p] if p >= 0 else self.c.host[self.hp[src, k], layer].numpy())[:rows]
        if idx_tail is not None:
            for pages in self.idx:
                a, b = pages[self.ix[src, k]], pages[idx_tail]
                b[:rows * 128] = a[:rows * 128]
                b[8192:8192 + 4 * rows] = a[8192:8192 + 4 * rows]
            self.ix[dst, k] = idx_tail
        self.bt[dst, k], self.hp[dst, k] = tail, -1

    def check(self):
        c = self.c
        n, width = self.bt.shape
        req = i32(range(n))
        bt, ix = (torch.full((n, width), 9, dtype=torch.int32, device="cuda") for _ in range(2))
        hp = torch.full((n, width), 9, dtype=torch.int64, device="cuda")
        c.pool.get_pages(req, 0, bt, ix, hp)
        for got, want in ((bt, self.bt), (ix, self.ix), (hp, self.hp)):
            assert np.array_equal(got.cpu().numpy(), want)
        for got, want in zip(c.kv, self.kv):
            assert np.array_equal(got.cpu().numpy().reshape(want.shape), want)
        for got, want in zip(c.idx, self.idx):
            assert np.array_equal(got.cpu().numpy(), want)


def spare(c):
    """Pool and index pages that no table names."""
    return ([p for p in range(c.n_pages) if not any(p in t for t in c.table)],
            [p for p in range(c.n_pages) if not any(p in t for t in c.idx_table)])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 700, 1280])
def test_one_fork(fmt, n):
    with Cache(pages=(20, 5), fmt=fmt, spare=2) as c:
        m = Model(c, 2)
        m.set_pages(0, 2, hp=[4, 5, 6])
        m.set_pages(0, 3, bt=[-1])                     # a placeholder stays one
        tail, idx_tail = (s[0] for s in spare(c))
        c.pool.fork_requests(i32([0]), i32([1]), i32([n]), i32([tail]), i32([idx_tail]))
        m.fork(0, 1, n, tail, idx_tail)
        assert c.pool.get_error() == 0
        m.check()


def test_many_forks_of_several_sources():
    """More table entries than one CTA has, forks that share a source, one without a last page, long and short."""
    lens = [1100 * 64 + 7, 64, 129, 5]
    with Cache(pages=(1101, 1, 3, 1) + (1,) * 9, n_layers=4, lpi=2, spare=12) as c:
        m = Model(c, 13)
        src = [0, 1, 2, 3, 0, 2, 0, 3, 1]
        n = [lens[s] for s in src]
        n[4] -= 500
        tail, idx_tail = (s[:9] for s in spare(c))
        c.pool.fork_requests(i32(src), i32(range(4, 13)), i32(n), i32(tail), i32(idx_tail))
        for k in range(9):
            m.fork(src[k], 4 + k, n[k], tail[k], idx_tail[k])
        assert c.pool.get_error() == 0
        m.check()


def test_a_fork_of_a_last_page_on_the_host_and_without_index_pages():
    with Cache(pages=(3, 1, 1), spare=3) as c:
        m = Model(c, 3)
        m.set_pages(0, 1, bt=[-1], hp=[3])
        tail, idx_tail = spare(c)
        c.pool.fork_requests(i32([0, 0]), i32([1, 2]), i32([100, 130]), i32(tail[:2]), i32(idx_tail[:2]))
        m.fork(0, 1, 100, tail[0], idx_tail[0])
        m.fork(0, 2, 130, tail[1], idx_tail[1])
        c.pool.fork_requests(i32([0]), i32([1]), i32([64 + 1]), i32([tail[2]]))
        m.fork(0, 1, 65, tail[2], None)
        assert c.pool.get_error() == 0
        m.check()


def test_forks_that_are_not_made():
    with Cache(pages=(4, 4, 1, 1, 1), spare=6) as c:
        m = Model(c, 5)
        m.set_pages(1, 1, bt=[-1])                     # neither here nor on the host
        t, ix = spare(c)
        for args, err in [(([-1], [2], [70], t[:1], ix[:1]), BAD_ID), (([5], [2], [70], t[:1], ix[:1]), BAD_ID),
                          (([0], [5], [70], t[:1], ix[:1]), BAD_ID), (([0], [-1], [70], t[:1], ix[:1]), BAD_ID),
                          (([0], [2], [-1], t[:1], ix[:1]), BAD_ID), (([0], [2], [c.max_ctx + 1], t[:1], ix[:1]), BAD_ID),
                          (([0], [0], [70], t[:1], ix[:1]), BAD_ID), (([0, 0], [2, 2], [70, 3], t[:2], ix[:2]), BAD_ID),
                          (([0], [2], [70], [c.n_pages], ix[:1]), BAD_ID), (([0], [2], [70], [-1], ix[:1]), BAD_ID),
                          (([0], [2], [70], t[:1], [c.n_pages]), BAD_ID), (([0], [2], [70], t[:1], [-1]), BAD_ID),
                          (([0, 0], [2, 3], [70, 71], [t[0]] * 2, ix[:2]), BAD_ID), (([0, 0], [2, 3], [70, 71], t[:2], [ix[0]] * 2), BAD_ID),
                          (([0], [2], [70], [int(c.table[0][1])], ix[:1]), BAD_ID),
                          (([0], [2], [70], t[:1], [int(c.idx_table[0][1])]), BAD_ID),
                          (([1], [2], [70], t[:1], ix[:1]), HOST_MISSING)]:
            c.pool.fork_requests(*[i32(a) for a in args])
            assert c.pool.get_error() == err, args
        m.check()
        # one bad fork among good ones; a chain of forks; the same tail where one of them does not use it
        c.pool.fork_requests(i32([0, 1, 0]), i32([2, 3, 4]), i32([70, 70, 128]), i32([t[0], t[1], t[0]]), i32([ix[0], ix[1], ix[0]]))
        assert c.pool.get_error() == HOST_MISSING
        m.fork(0, 2, 70, t[0], ix[0])
        m.fork(0, 4, 128, t[0], ix[0])
        m.check()
        c.pool.fork_requests(i32([0, 2]), i32([2, 3]), i32([70, 70]), i32(t[2:4]), i32(ix[2:4]))
        assert c.pool.get_error() == BAD_ID            # 2 is a destination and a source: only 2 -> 3 is made
        m.fork(2, 3, 70, t[3], ix[3])
        m.check()
        c.pool.fork_requests(i32([]), i32([]), i32([]), i32([]), i32([]))
        lib, st, p = c.H.lib, torch.cuda.current_stream().cuda_stream, i32([0] * 8).data_ptr()
        assert lib.hs_fork_requests(c.pool.handle, 6, p, p, p, p, p, st) == INVALID       # more than requests
        assert lib.hs_fork_requests(c.pool.handle, -1, p, p, p, p, p, st) == INVALID
        for k in range(5):
            for at in (None, p + 2):
                if at is None and k == 4:
                    continue
                a = [p] * 5
                a[k] = at
                assert lib.hs_fork_requests(c.pool.handle, 1, *a, st) == INVALID, (k, at)
        m.check()


def moved(m, kind, src, dst, remap):
    tables, pages = ((m.bt,), m.kv) if kind == "kv" else ((m.ix,), m.idx)
    for p in pages:
        p[dst] = p[src].copy()
    if remap:
        now = np.arange(m.c.n_pages)
        now[src] = dst
        for t in tables:
            t[t >= 0] = now[t[t >= 0]]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("remap", [False, True])
@pytest.mark.parametrize("n,layers,lpi", [(1, 1, 1), (5, 3, 2), (300, 2, 2), (700, 1, 1)])
def test_copies_and_moves(fmt, remap, n, layers, lpi):
    with Cache(n_layers=layers, lpi=lpi, pages=(n // 2 + 1, n // 2 + 2, 3), fmt=fmt, spare=n + 3) as c:
        m = Model(c, 3)
        m.set_pages(2, 0, bt=list(c.table[0][:2]))     # pages that two requests share
        rng = np.random.default_rng(n)
        free, idx_free = spare(c)
        src, idx_src = rng.permutation(np.concatenate(c.table[:2]))[:n], rng.permutation(np.concatenate(c.idx_table))[:n // 2 + 1]
        dst, idx_dst = np.array(free)[:n], np.array(idx_free)[-len(idx_src):]
        c.pool.copy_pages(i32(src), i32(dst), i32(idx_src), i32(idx_dst), remap=remap)
        moved(m, "kv", src, dst, remap)
        moved(m, "idx", idx_src, idx_dst, remap)
        assert c.pool.get_error() == 0
        m.check()
        # one kind alone, back again
        c.pool.copy_pages(i32(dst), i32(src), remap=remap)
        moved(m, "kv", dst, src, remap)
        c.pool.copy_pages(idx_src=i32(idx_dst), idx_dst=i32(idx_src), remap=remap)
        moved(m, "idx", idx_dst, idx_src, remap)
        assert c.pool.get_error() == 0
        m.check()


def test_the_most_pages_of_a_call():
    n = 4096
    with Cache(n_layers=1, lpi=1, pages=(n, 2), spare=n, host_pages=1) as c:
        m = Model(c, 2)
        src, dst = c.table[0], np.array(spare(c)[0])[:n]
        isrc, idst = c.idx_table[0], np.array(spare(c)[1])[:n]
        c.pool.copy_pages(i32(src), i32(dst), i32(isrc), i32(idst), remap=True)
        moved(m, "kv", src, dst, True)
        moved(m, "idx", isrc, idst, True)
        assert c.pool.get_error() == 0
        m.check()
        with pytest.raises(c.H.HisparseError):
            c.pool.copy_pages(i32([0] * (n + 1)), i32([1] * (n + 1)))


def test_copies_that_are_not_made():
    """A destination named twice, a destination that is a source, a page onto itself, ids out of range, a
    source moved twice; the other copies of the call are made. A source copied to two places is fine."""
    with Cache(pages=(6, 2), spare=8, n_layers=2) as c:
        m = Model(c, 2)
        t, f = [int(x) for x in c.table[0]], spare(c)[0]
        good = ([t[4]], [f[6]])
        for src, dst in [([t[0], t[1]], [f[0], f[0]]), ([t[0]], [t[0]]), ([-1], [f[0]]), ([c.n_pages], [f[0]]), ([t[0]], [-1]),
                         ([t[0]], [c.n_pages]), ([t[0], t[0]], [f[0], f[0]])]:
            for remap in (False, True):
                c.pool.copy_pages(i32(src + good[0]), i32(dst + good[1]), remap=remap)
                assert c.pool.get_error() == BAD_ID, (src, dst)
                moved(m, "kv", np.array(good[0]), np.array(good[1]), remap)
                m.check()
                if remap:
                    good = (good[1], good[0])
        # a chain: the copy onto a source is not made, the copy from it is
        c.pool.copy_pages(i32([t[0], t[1]]), i32([t[1], f[0]]))
        assert c.pool.get_error() == BAD_ID
        moved(m, "kv", np.array([t[1]]), np.array([f[0]]), False)
        m.check()
        c.pool.copy_pages(i32([t[0], t[0]]), i32([f[1], f[2]]))
        assert c.pool.get_error() == 0
        moved(m, "kv", np.array([t[0], t[0]]), np.array([f[1], f[2]]), False)
        m.check()
        c.pool.copy_pages(i32([t[0], t[0]]), i32([f[3], f[4]]), remap=True)
        assert c.pool.get_error() == BAD_ID
        m.check()
        c.pool.copy_pages(idx_src=i32([-5]), idx_dst=i32([0]), remap=True)
        assert c.pool.get_error() == BAD_ID
        c.pool.copy_pages()
        c.pool.copy_pages(i32([]), i32([]), remap=True)
        assert c.pool.get_error() == 0
        m.check()
        lib, st, p = c.H.lib, torch.cuda.current_stream().cuda_stream, i32([0] * 8).data_ptr()
        for a in [(-1, p, p, 0, None, None), (1, None, p, 0, None, None), (1, p, None, 0, None, None), (1, p + 1, p, 0, None, None),
                  (1, p, p + 2, 0, None, None), (0, None, None, 1, None, p), (0, None, None, 1, p, p + 2), (0, None, None, 4097, p, p)]:
            assert lib.hs_copy_pages(c.pool.handle, *a, 0, st) == INVALID, a


@pytest.mark.parametrize("remap", [False, True])
@pytest.mark.parametrize("n,n_idx", [(63, 1), (64, 64), (65, 64), (64, 65), (0, 64), (64, 0), (1, 66)])
def test_copies_around_the_number_that_are_checked_beside_the_copying(n, n_idx, remap):
    """Of both kinds, with a copy in each list that is not made: the last one has the first one's source as its destination."""
    with Cache(n_layers=2, lpi=1, pages=(80, 3), spare=80) as c:
        m = Model(c, 2)
        m.set_pages(1, 0, bt=list(c.table[0][:2]))
        for kind, k in (("kv", n), ("idx", n_idx)):
            free = spare(c)[0 if kind == "kv" else 1]
            src = np.random.default_rng(k).permutation((c.table if kind == "kv" else c.idx_table)[0])[:k]
            dst = np.array(free)[:k]
            made = np.ones(k, bool)
            if k > 1:
                dst[-1], made[-1] = src[0], False
            if kind == "kv":
                kv = (src, dst, made)
            else:
                idx = (src, dst, made)
        c.pool.copy_pages(i32(kv[0]), i32(kv[1]), i32(idx[0]), i32(idx[1]), remap=remap)
        for kind, (src, dst, made) in (("kv", kv), ("idx", idx)):
            moved(m, kind, src[made], dst[made], remap)
        assert c.pool.get_error() == BAD_ID
        m.check()


def test_a_moved_hot_page_keeps_its_rows():
    """A missed row lies in a hot buffer; after its page has moved, a replay finds it in the new place."""
    with Cache(pages=(8, 1), n_layers=2, lpi=2, spare=6, heads=16) as c:
        m = Model(c, 2)
        free = spare(c)[0]
        m.set_pages(0, 2, bt=[-1], hp=[5])             # page 2 of request 0 is on the host alone
        c.pool.hot_lease(0, 0, [free[0]])
        topk = torch.full((1, 128), -1, dtype=torch.int32, device="cuda")
        topk[0, :3] = i32([5, 130, 200])
        rows, again = torch.empty(1, 128, dtype=torch.int32, device="cuda"), torch.empty(1, 128, dtype=torch.int32, device="cuda")
        c.pool.resolve_topk(0, 1, i32([0]), topk, rows)
        assert c.pool.get_error() == 0
        hot = int(rows[0, 1])
        assert hot // 64 == free[0]
        c.pool.copy_pages(i32([free[0], int(c.table[0][0])]), i32([free[1], free[2]]), remap=True)
        c.pool.replay_topk(0, i32([0]), topk, again)
        assert c.pool.get_error() == 0
        want = rows.clone()
        want[0, 0] = free[2] * 64 + 5
        want[0, 1] = free[1] * 64 + hot % 64
        assert torch.equal(again, want)
        for layer in range(2):
            assert np.array_equal(c.kv[layer][int(again[0, 1])].cpu().numpy(), c.host[5, layer, 2].numpy())


def test_tables_read_back_in_part():
    with Cache(pages=(7, 4, 9)) as c:
        m = Model(c, 3)
        got = torch.full((4, 3), 77, dtype=torch.int32, device="cuda")
        c.pool.get_pages(i32([2, 0, 2, 1]), 2, got)
        assert np.array_equal(got.cpu().numpy(), m.bt[[2, 0, 2, 1], 2:5]) and c.pool.get_error() == 0
        host = torch.full((2, 1), 77, dtype=torch.int64, device="cuda")
        c.pool.get_pages(i32([3, 1]), 0, host_pages=host)
        assert host.cpu().tolist() == [[-1], [-1]] and c.pool.get_error() == BAD_ID
        width = c.max_ctx // 64
        for first, n in ((-1, 2), (width, 1), (width - 1, 2)):
            with pytest.raises(c.H.HisparseError):
                c.pool.get_pages(i32([0]), first, torch.zeros(1, n, dtype=torch.int32, device="cuda"))
        c.pool.get_pages(i32([]), 0, torch.zeros(0, 3, dtype=torch.int32, device="cuda"))


def test_a_fork_of_the_longest_context():
    """Every table entry of a context as long as a pool takes, over several CTAs."""
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    with Cache(n_layers=1, lpi=1, pages=(3, 1), max_ctx=H.MAX_CTX, host_pages=5) as c:
        m = Model(c, 2)
        rng = np.random.default_rng(3)
        n = H.MAX_CTX // 64
        m.set_pages(0, 0, bt=rng.integers(-1, c.n_pages, n).tolist(), ix=rng.integers(-1, c.n_pages, n).tolist(),
                    hp=rng.integers(-1, 5, n).tolist())
        tail, idx_tail = (s[0] for s in spare(c))
        for length in (H.MAX_CTX, 64 * (n - 1), 64 * 1024, 64 * 1023):
            c.pool.fork_requests(i32([0]), i32([1]), i32([length]), i32([tail]), i32([idx_tail]))
            m.fork(0, 1, length, tail, idx_tail)
            assert c.pool.get_error() == 0
            m.check()
