"""Through which request's table a group's shared pages are read, and ragged groups of 32 heads that share."""
import numpy as np
import pytest

from test_gpu_cache_ops import HOST_MISSING, check_chunk, make_q, torch
from test_gpu_prefix import SM, Shared, layout, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", ["nothing", "bad"])
def test_the_reader_is_the_first_segment_that_has_tokens(first):
    """The group's first segment has none, and its request no rows, or is none: the second one's table is read."""
    lengths = [700 + i for i in range(13)]
    with Shared(16, [13], [640], lengths) as s:
        c = s.c
        news = [0] + [1] * 12
        start, limit = layout(news, lengths)
        c.pool.set_pages(0, 0, block_table=[-1] * 10, host_pages=[-1] * 10)
        q = make_q(s.rng, 12, 16, "bf16")
        req = ([0] if first == "nothing" else [-1]) + list(range(1, 13))
        out, lse = run(c, [0, 13], [640], req, start, limit, q)
        assert c.pool.get_error() == 0
        check_chunk(c, s.kv, list(range(13)), start, limit, q, SM, out, lse, "bf16")
        # the second one's is: without its first page, that is seen by none of the twelve
        c.pool.set_pages(1, 0, block_table=[-1], host_pages=[-1])
        out, lse = run(c, [0, 13], [640], req, start, limit, q)
        assert c.pool.get_error() == HOST_MISSING
        gone = [np.delete(k, slice(0, 64), 0) for k in s.kv]
        check_chunk(c, gone, list(range(13)), start, limit - 64, q, SM, out, lse, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ragged_groups_of_32_heads(dtype):
    """Segments of one to seven tokens, whose blocks of four are partly empty where each reads alone and full where they
    share, behind prefixes of whole and of partly filled pages; limits within and at the end of what is shared. Twice,
    bit for bit."""
    sizes, prefix = [7, 1, 11, 3], [2048, 0, 1300, 64]
    rng = np.random.default_rng(3)
    lengths = [max(8, prefix[g]) + int(rng.integers(8, 300)) for g, k in enumerate(sizes) for _ in range(k)]
    news = [1, 3, 2, 5, 1, 7, 2, 6] + [1, 1, 2, 3, 1, 5, 1, 1, 2, 1, 6] + [1, 2, 3]
    with Shared(32, sizes, prefix, lengths, copies=False) as s:
        start, limit = layout(news, lengths, lead=1, tail=2)
        a = start[5]
        limit[a:a + 7] = [0, 1, 2048, 2047, 1985, 64, 65]
        limit[start[10]:start[10] + 2] = [1280, 1281]
        q = make_q(s.rng, len(limit), 32, dtype)
        out, lse = run(s.c, s.group_start, s.group_len, range(len(lengths)), start, limit, q)
        again, l2 = run(s.c, s.group_start, s.group_len, range(len(lengths)), start, limit, q)
        assert s.c.pool.get_error() == 0 and torch.equal(out, again) and torch.equal(lse, l2)
        check_chunk(s.c, s.kv, range(len(lengths)), start, limit, q, SM, out, lse, dtype)


@pytest.mark.parametrize("heads,k,pages", [(16, 2, (5, 6, 7)), (64, 4, (13, 14, 15)), (32, 12, (4, 5))])
def test_groups_next_to_the_border_of_sharing(heads, k, pages):
    """What is saved is a little less than what sharing costs, as much, and a little more."""
    for p in pages:
        lengths = [64 * p + 1 + (i * 37) % 90 for i in range(3 * k)]
        with Shared(heads, [k] * 3, [64 * p] * 3, lengths, seed=p) as s:
            start, limit = layout([1] * (3 * k), lengths)
            q = make_q(s.rng, 3 * k, heads, "bf16")
            out, lse = run(s.c, s.group_start, s.group_len, range(3 * k), start, limit, q)
            assert s.c.pool.get_error() == 0
            check_chunk(s.c, s.kv, range(3 * k), start, limit, q, SM, out, lse, "bf16")


@pytest.mark.parametrize("heads,tokens", [(64, 12), (64, 13), (16, 48), (16, 49), (16, 64), (16, 65)])
def test_joins_next_to_the_border_of_rows(heads, tokens):
    """Rows joined by slices and without, of parts of many pairs."""
    lengths = [3000 + i for i in range(tokens)]
    with Shared(heads, [tokens], [2944], lengths, seed=tokens) as s:
        start, limit = layout([1] * tokens, lengths)
        q = make_q(s.rng, tokens, heads, "bf16")
        out, lse = run(s.c, s.group_start, s.group_len, range(tokens), start, limit, q)
        again, l2 = run(s.c, s.group_start, s.group_len, range(tokens), start, limit, q)
        assert s.c.pool.get_error() == 0 and torch.equal(out, again) and torch.equal(lse, l2)
        check_chunk(s.c, s.kv, range(tokens), start, limit, q, SM, out, lse, "bf16", set(range(0, tokens, 5)) | {tokens - 1})
