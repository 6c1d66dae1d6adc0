"""Rotations of more tokens than a decode has, straight before calls that read their queries before they wait for the
kernel in front of them: a prefill chunk whose requests decode beside it is rotated in one call."""
import math

import numpy as np
import pytest

from cache_plain import pack_rows
from test_gpu_cache_ops import Cache, i32, make_q, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1025, 4099])
def test_queries_of_a_mixed_batch_rotated_straight_before_the_sparse_attention(n):
    """The decode's queries are the last two tokens, and the first two, of a larger rotation; every pass of a graph has
    other values for them, so that queries of the pass before would show."""
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    heads, passes = 64, 6
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(8,), seed=1) as c:
        rng = np.random.default_rng(n)
        c.put_rows(0, 0, np.arange(512), pack_rows(rng.standard_normal((512, 512)), rng.standard_normal((512, 64))))
        ids = torch.from_numpy(c.rows_at(0, np.arange(128)).astype(np.int32)).cuda()[None].repeat(2, 1)
        steps, _ = H.rotary_steps(64, 10000.0)
        steps, pos = steps.cuda(), i32(np.arange(n) + 777)
        x = make_q(rng, n, heads, "bf16")
        qs = [x * (0.5 + k) for k in range(passes)]
        buf = torch.zeros(n, heads, 576, dtype=torch.bfloat16, device="cuda")
        outs = [[torch.zeros(2, heads, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in qs]

        def rotate(q):
            c.pool.rotary(pos, steps, [(q[:, :, 512:], buf[:, :, 512:], "halves"), (q[:, :, :64], buf[:, :, :64], "pairs")])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for q, (last, first) in zip(qs, outs):
                rotate(q)
                c.pool.sparse_mla_decode(0, buf[n - 2:], ids, 1 / math.sqrt(576), last)
                rotate(q)
                c.pool.sparse_mla_decode(0, buf[:2], ids, 1 / math.sqrt(576), first)
        for _ in range(20):
            g.replay()
        torch.cuda.synchronize()
        for q, found in zip(qs, outs):
            rotate(q)
            torch.cuda.synchronize()
            for part, out in zip((buf[n - 2:], buf[:2]), found):
                want = torch.zeros_like(out)
                c.pool.sparse_mla_decode(0, part, ids, 1 / math.sqrt(576), want)
                torch.cuda.synchronize()
                assert torch.equal(out, want)
        assert c.pool.get_error() == 0
