"""Calls that read tables or queries before they wait for the kernel in front of them, straight behind the calls
that write these: every row lands, and every query is read, as if each call had been waited for."""
import numpy as np
import pytest

from test_gpu_cache_ops import Cache, i32, make_q, torch

pytestmark = pytest.mark.gpu


def test_rows_appended_straight_behind_forks_and_moves():
    """40 forks of one request with last pages in turn, each followed by an append to that page, and moves of the
    source's last page in between, to which is appended at once, replayed as one graph."""
    with Cache(n_layers=2, lpi=2, pages=(2, 1), spare=6, fmt=0) as c:
        rng = np.random.default_rng(0)
        free = [p for p in range(c.n_pages) if not any(p in t for t in c.table)]
        ifree = [p for p in range(c.n_pages) if not any(p in t for t in c.idx_table)]
        c.pool.set_pages(1, 0, block_table=[-1], idx_pages=[-1])
        n = 40
        rows = torch.from_numpy(rng.integers(0, 256, (n, 1, 2, 656), dtype=np.uint8)).cuda()
        keys = torch.from_numpy(rng.integers(-127, 128, (n, 1, 1, 128)).astype(np.int8)).cuda()
        ids = [[i32([0]), i32([1]), i32([70]), i32([free[k % 3]]), i32([ifree[k % 3]])] for k in range(n)]
        pos = [i32([70 + k % 50]) for k in range(n)]
        one = i32([1])
        home = int(c.table[0][1])
        away = [i32([home]), i32([free[3]])]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for k in range(n):
                c.pool.fork_requests(*ids[k])
                c.pool.append_rows(one, pos[k], rows[k], keys[k])
                c.pool.copy_pages(*(away if k % 2 == 0 else away[::-1]), remap=True)
                c.pool.append_rows(ids[k][0], pos[k], rows[k], keys[k])
        for _ in range(20):
            for t in c.kv:
                t.fill_(1)
            g.replay()
            torch.cuda.synchronize()
            assert c.pool.get_error() == 0
            want = np.ones((c.n_pages, 64, 656), np.uint8)
            for k in range(n):
                tail, at, to = want[free[k % 3]], home if k % 2 == 0 else free[3], free[3] if k % 2 == 0 else home
                tail[:6] = want[at][:6]
                p = 6 + k % 50
                tail[p] = rows[k, 0, 1].cpu().numpy()
                want[to] = want[at]
                want[to][p] = rows[k, 0, 1].cpu().numpy()
            assert np.array_equal(c.kv[1].cpu().numpy().reshape(want.shape), want)


def test_queries_rotated_straight_before_the_sparse_attention():
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    with Cache(heads=64, n_layers=1, lpi=1, pages=(8,), seed=1) as c:
        rng = np.random.default_rng(1)
        from cache_plain import pack_rows
        c.put_rows(0, 0, np.arange(512), pack_rows(rng.standard_normal((512, 512)), rng.standard_normal((512, 64))))
        ids = torch.from_numpy(c.rows_at(0, np.arange(128)).astype(np.int32)).cuda()[None]
        steps, _ = H.rotary_steps(64, 10000.0)
        steps = steps.cuda()
        qs = [make_q(rng, 1, 64, "bf16") for _ in range(24)]
        buf, pos = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda"), i32([12345])
        outs = [torch.zeros(1, 64, 512, dtype=torch.bfloat16, device="cuda") for _ in qs]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for q, out in zip(qs, outs):
                c.pool.rotary(pos, steps, [(q[:, :, 512:], buf[:, :, 512:], "halves"), (q[:, :, :64], buf[:, :, :64], "pairs")])
                c.pool.sparse_mla_decode(0, buf, ids, 0.04, out)
        for _ in range(20):
            g.replay()
        torch.cuda.synchronize()
        for q, out in zip(qs, outs):
            c.pool.rotary(pos, steps, [(q[:, :, 512:], buf[:, :, 512:], "halves"), (q[:, :, :64], buf[:, :, :64], "pairs")])
            torch.cuda.synchronize()
            want = torch.zeros_like(out)
            c.pool.sparse_mla_decode(0, buf, ids, 0.04, want)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert c.pool.get_error() == 0
