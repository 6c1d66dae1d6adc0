"""Attention of requests that share their first positions, on the GPU against the plain 64-bit attention of
each token over its own request, within the bounds of the attention it is built on."""
import math

import numpy as np
import pytest

import cache_plain as CP
from test_gpu_cache_ops import BAD_ID, HOST_MISSING, INVALID, RANGE, Cache, check_chunk, i32, make_q, torch

pytestmark = pytest.mark.gpu
SM = 1 / math.sqrt(576)


class Shared:
    """Requests in groups: group g has sizes[g] requests whose first prefix[g] positions hold the same rows
    (whole pages shared, the rest copied); request r has lengths[r] positions. Bytes of no row are 0xFF."""

    def __init__(self, heads, sizes, prefix, lengths, seed=0, copies=False, **more):
        of = [g for g, k in enumerate(sizes) for _ in range(k)]
        start = np.r_[0, np.cumsum(sizes)]
        assert len(lengths) == len(of)
        kept = [0 if r == start[g] or copies else min(prefix[g], n) // 64 for r, (n, g) in enumerate(zip(lengths, of))]
        pages = [max(1, -(-n // 64) - k) for n, k in zip(lengths, kept)]
        self.c = c = Cache(heads=heads, n_layers=2, lpi=2, pages=pages, max_ctx=-(-max(lengths) // 128) * 128, **more)
        rng = self.rng = np.random.default_rng(seed)
        self.kv, rows_of = [], {}
        for r, (n, g) in enumerate(zip(lengths, of)):
            first = int(start[g])
            same = 0 if r == first else min(prefix[g], n, lengths[first])
            if kept[r]:
                c.table[r] = np.r_[c.table[first][:kept[r]], c.table[r]]
                c.pool.set_pages(r, 0, block_table=list(c.table[r][:-(-n // 64)]))
            x = rng.standard_normal((n - same, 576)) * np.exp(0.3 * rng.standard_normal((n - same, 1)))
            rows = CP.pack_rows(x[:, :512], x[:, 512:]) if n > same else np.zeros((0, 656), np.uint8)
            values = CP.row_values(rows)
            if same:
                rows, values = np.r_[rows_of[g][0][:same], rows], np.r_[rows_of[g][1][:same], values]
            if r == first:
                rows_of[g] = rows, values
            if n > kept[r] * 64:
                c.put_rows(1, r, np.arange(kept[r] * 64, n), rows[kept[r] * 64:])
            self.kv.append(values)
        self.group_start, self.group_len = start, np.array(prefix)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.c.__exit__(*a)


def run(c, group_start, group_len, seg_req, seg_start, limit, q, sm=SM, out=None, lse=True, work=None, stream=None, layer=1):
    n = q.shape[0]
    out = torch.full((n, c.heads, 512), 0.25, dtype=q.dtype, device="cuda") if out is None else out
    l = torch.full((n, c.heads), 0.25, device="cuda") if lse else None
    if work is None:
        work = torch.full((c.pool.prefix_workspace_bytes(n, len(seg_req), len(group_len)),), 255, dtype=torch.uint8, device="cuda")
    c.pool.prefix_attention(layer, i32(group_start), i32(group_len), i32(seg_req), i32(seg_start), i32(limit), q, sm, out, work, lse=l,
                            stream=stream)
    return out, l


def layout(news, lengths, lead=0, tail=0):
    """Starts and limits of segments whose last token sees their request's whole length."""
    start = lead + np.r_[0, np.cumsum(news)]
    limit = np.zeros(int(start[-1]) + tail, np.int64)
    for i, (m, n) in enumerate(zip(news, lengths)):
        limit[start[i]:start[i + 1]] = np.arange(n - m + 1, n + 1)
    return start, limit


@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_groups_of_single_tokens(heads, dtype):
    """Groups of 1 to 40 requests, prefixes of whole and of partly filled pages, shorter than one, and none."""
    sizes, prefix = [12, 1, 5, 40, 3, 2], [640, 0, 700, 64, 63, 1000]
    rng = np.random.default_rng(heads)
    lengths = [prefix[g] + int(rng.integers(1, 200)) for g, k in enumerate(sizes) for _ in range(k)]
    with Shared(heads, sizes, prefix, lengths) as s:
        start, limit = layout([1] * len(lengths), lengths, lead=2, tail=3)
        q = make_q(s.rng, len(limit), heads, dtype)
        out, lse = run(s.c, s.group_start, s.group_len, range(len(lengths)), start, limit, q)
        assert s.c.pool.get_error() == 0
        check_chunk(s.c, s.kv, range(len(lengths)), start, limit, q, SM, out, lse, dtype)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("copies", [False, True])
def test_ragged_segments_and_limits(heads, copies):
    """Segments of 0 to 70 tokens, limits out of order, within the prefix, at its end and 0; segments in front
    of, between and behind the groups; a long prefix whose blocks several pairs cut."""
    sizes, prefix = [1, 9, 1, 6, 2], [0, 4160, 0, 333, 256]
    lengths = [70, 4161, 4200, 4160, 5000, 4300, 4170, 4180, 4190, 4230, 129, 400, 334, 340, 500, 600, 333, 256, 300]
    news = [3, 1, 9, 2, 70, 0, 4, 4, 1, 30, 65, 5, 1, 7, 64, 4, 3, 1, 6]
    with Shared(heads, sizes, prefix, lengths, copies=copies) as s:
        start, limit = layout(news, lengths, lead=1, tail=2)
        a = start[4]
        limit[a:a + 70] = s.rng.permutation(limit[a:a + 70])
        limit[a + 3], limit[a + 4], limit[a + 5], limit[a + 6], limit[a + 7] = 0, 1, 4160, 4096, 2000
        limit[start[14]:start[14] + 64] = s.rng.integers(0, 334, 64)       # a segment within its prefix
        limit[start[18]:start[19]] = 0                                       # and one that sees nothing
        q = make_q(s.rng, len(limit), heads, "bf16")
        q[start[18]:start[19]] = float("nan")
        groups = np.r_[1, 10, 11, 17, 19]                                    # the first segment is of no group
        out, lse = run(s.c, groups, [4160, 0, 333, 256], range(len(lengths)), start, limit, q)
        assert s.c.pool.get_error() == 0
        q[start[18]:start[19]] = 0
        some = set(range(0, len(limit), 3)) | set(range(a, a + 9)) | set(range(start[17], start[19]))
        check_chunk(s.c, s.kv, range(len(lengths)), start, limit, q, SM, out, lse, "bf16", some)


def test_no_groups_and_groups_that_gain_nothing():
    """What is not shared is read by each segment alone (the ranges of pages, and so the order of sums, may differ
    from chunk_attention's)."""
    lengths = [200, 300, 70, 1000]
    with Shared(64, [2, 2], [128, 64], lengths) as s:
        start, limit = layout([2, 2, 2, 2], lengths)     # blocks of 64 heads hold two tokens: nothing to gain
        q = make_q(s.rng, 8, 64, "bf16")
        for groups, lens in (([0], []), ([0, 2, 4], [128, 64]), ([0, 0, 4], [128, 0]), ([1, 2], [128])):
            out, lse = run(s.c, groups, lens, range(4), start, limit, q)
            assert s.c.pool.get_error() == 0
            check_chunk(s.c, s.kv, range(4), start, limit, q, SM, out, lse, "bf16")


@pytest.mark.parametrize("heads,tokens", [(16, 600), (64, 150)])
def test_long_prefixes_and_many_blocks(heads, tokens):
    """More shared blocks than pairs of SMs hold, with more rows than the wide join takes; twice, bit for bit."""
    p = 20032
    lengths = [p + 1 + (i * 37) % 300 for i in range(tokens)]
    with Shared(heads, [tokens], [p], lengths) as s:
        start, limit = layout([1] * tokens, lengths)
        q = make_q(s.rng, tokens, heads, "bf16")
        out, lse = run(s.c, s.group_start, s.group_len, range(tokens), start, limit, q)
        again, l2 = run(s.c, s.group_start, s.group_len, range(tokens), start, limit, q)
        assert s.c.pool.get_error() == 0 and torch.equal(out, again) and torch.equal(lse, l2)
        check_chunk(s.c, s.kv, range(tokens), start, limit, q, SM, out, lse, "bf16", set(range(0, tokens, 97)) | {tokens - 1})


def test_strides_and_no_lse():
    lengths = [700 + i for i in range(20)]
    with Shared(32, [20], [640], lengths) as s:
        start, limit = layout([1] * 20, lengths)
        wide = make_q(s.rng, 20, 33, "fp16")
        big = torch.full((20, 40, 520), 0.25, dtype=torch.float16, device="cuda")
        q, out = wide[:, 1:], big[:, 8:, :512]
        run(s.c, s.group_start, s.group_len, range(20), start, limit, q, out=out, lse=False)
        want, wl = run(s.c, s.group_start, s.group_len, range(20), start, limit, q.contiguous())
        assert torch.equal(out, want) and torch.all(big[:, :8] == 0.25) and torch.all(big[:, :, 512:] == 0.25)
        check_chunk(s.c, s.kv, range(20), start, limit, q, SM, want, wl, "fp16")


def test_bad_groups_lengths_and_requests():
    """What is clamped reads each segment's own rows and stays right; a bad request sees nothing."""
    lengths = [700 + i for i in range(24)]
    with Shared(16, [12, 12], [640, 640], lengths) as s:
        c = s.c
        start, limit = layout([1] * 24, lengths)
        q = make_q(s.rng, 24, 16, "bf16")
        every = list(range(24))
        for groups, lens in (([0, 12, 30], [640, 640]), ([-3, 12, 24], [640, 640]), ([0, 12, 5], [640, 640]), ([0, 12, 24], [-1, 640]),
                             ([0, 12, 24], [640, c.max_ctx + 1])):
            out, lse = run(c, groups, lens, every, start, limit, q)
            assert c.pool.get_error() == BAD_ID, (groups, lens)
            check_chunk(c, s.kv, every, start, limit, q, SM, out, lse, "bf16")
        for bad in (-1, 24):
            req = list(every)
            req[4] = bad
            out, lse = run(c, [0, 12, 24], [640, 640], req, start, limit, q)
            assert c.pool.get_error() == BAD_ID
            assert not out[4].any() and torch.all(torch.isneginf(lse[4]))
            out[4], lse[4] = out[5], lse[5]
            check_chunk(c, s.kv, every, start, limit, q, SM, out, lse, "bf16", set(every) - {4})
        lim = limit.copy()
        lim[3], lim[20] = -1, c.max_ctx + 1
        out, lse = run(c, [0, 12, 24], [640, 640], every, start, lim, q)
        assert c.pool.get_error() == BAD_ID
        for j in (3, 20):
            assert not out[j].any() and torch.all(torch.isneginf(lse[j]))
        check_chunk(c, s.kv, every, start, limit, q, SM, out, lse, "bf16", set(every) - {3, 20})


def test_shared_pages_on_the_host_and_missing():
    lengths = [300 + i for i in range(16)]
    with Shared(16, [16], [256], lengths) as s:
        c = s.c
        start, limit = layout([1] * 16, lengths)
        q = make_q(s.rng, 16, 16, "bf16")
        c.host[2, 1] = c.kv[1].view(-1, 64, 656)[int(c.table[0][1])].cpu()
        c.pool.set_pages(0, 1, block_table=[-1], host_pages=[2])       # of the request that the group is read through
        out, lse = run(c, s.group_start, s.group_len, range(16), start, limit, q)
        assert c.pool.get_error() == 0
        check_chunk(c, s.kv, range(16), start, limit, q, SM, out, lse, "bf16")
        c.pool.set_pages(0, 1, host_pages=[-1])
        out, lse = run(c, s.group_start, s.group_len, range(16), start, limit, q)
        assert c.pool.get_error() == HOST_MISSING
        gone = [np.delete(k, slice(64, 128), 0) for k in s.kv]         # counts as not seen
        check_chunk(c, gone, range(16), start, limit - 64, q, SM, out, lse, "bf16")


def test_values_beyond_the_range():
    """A row that is not finite in the shared part, queries that are not, scores far below: reported, and not seen."""
    lengths = [200 + i for i in range(16)]
    with Shared(16, [16], [192], lengths) as s:
        c = s.c
        start, limit = layout([1] * 16, lengths)
        q = make_q(s.rng, 16, 16, "bf16")
        bad = c.get_rows(1, 0, [70])
        good = bad.copy()
        bad[0, 528 + 4:528 + 6] = [0xC0, 0x7F]                           # a NaN in the rope of position 70
        c.put_rows(1, 0, [70], bad)
        q[5, 3, 17] = float("inf")
        out, lse = run(c, s.group_start, s.group_len, range(16), start, limit, q)
        assert c.pool.get_error() == RANGE
        assert not out[5, 3].any() and torch.isneginf(lse[5, 3])
        q[5, 3, 17] = 0
        gone = [np.delete(k, 70, 0) for k in s.kv]
        check_chunk(c, gone, range(16), start, limit - 1, q, SM, out, lse, "bf16", set(range(16)) - {5})
        c.put_rows(1, 0, [70], good)
        # every score of the shared part below the range, those behind it within: weights of the latter alone
        big = torch.zeros(16, 16, 576, dtype=torch.bfloat16, device="cuda")
        big[:, :, 575] = 60000.0
        rows = c.get_rows(1, 0, np.arange(192))
        rows[:, 654:656] = np.frombuffer(np.array([0xC2C8], "<u2").tobytes(), np.uint8)
        c.put_rows(1, 0, np.arange(192), rows)                           # rope 63 of the shared rows: -100
        kv = []
        for r, n in enumerate(lengths):
            mine = c.get_rows(1, r, np.arange(192, n))
            mine[:, 654:656] = 0
            c.put_rows(1, r, np.arange(192, n), mine)
            kv.append(CP.row_values(mine))                               # the shared rows weigh nothing
        out, lse = run(c, s.group_start, s.group_len, range(16), start, limit, big, sm=1.0)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, range(16), start, limit - 192, big, 1.0, out, lse, "bf16")
        # and of all of a token's parts: sees nothing, and is reported
        for r, n in enumerate(lengths):
            mine = c.get_rows(1, r, np.arange(192, n))
            mine[:, 654:656] = np.frombuffer(np.array([0xC2C8], "<u2").tobytes(), np.uint8)
            c.put_rows(1, r, np.arange(192, n), mine)
        out, lse = run(c, s.group_start, s.group_len, range(16), start, limit, big, sm=1.0)
        assert c.pool.get_error() == RANGE
        assert not out.any() and torch.all(torch.isneginf(lse))


def test_refusals_and_empty_calls():
    lengths = [130] * 4
    with Shared(16, [4], [128], lengths) as s:
        c = s.c
        H, lib, st = c.H, c.H.lib, torch.cuda.current_stream().cuda_stream
        q = make_q(s.rng, 4, 16, "bf16")
        out = torch.full((4, 16, 512), 0.25, dtype=torch.bfloat16, device="cuda")
        ids = i32([0, 1, 2, 3, 4, 130, 130, 130, 130, 0, 4, 128])
        at = ids.data_ptr()
        need = c.pool.prefix_workspace_bytes(4, 4, 1)
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        ok = dict(layer=1, groups=1, gs=at + 36, gl=at + 44, segs=4, sr=at, ss=at, n=4, lim=at + 20, dtype=0, q=q.data_ptr(),
                  qt=9216, qh=576, sm=SM, out=out.data_ptr(), ot=8192, oh=512, lse=None, work=work.data_ptr(), bytes=need)

        def call(**bad):
            a = {**ok, **bad}
            return lib.hs_prefix_attention(c.pool.handle, *list(a.values())[:13], *list(a.values())[13:], st)

        for bad in [dict(layer=2), dict(layer=-1), dict(groups=-1), dict(groups=2049), dict(gs=None), dict(gl=None), dict(gs=at + 2),
                    dict(gl=at + 1), dict(segs=-1), dict(segs=4097), dict(n=-1), dict(n=16385), dict(dtype=2), dict(sr=None),
                    dict(ss=at + 2), dict(lim=None), dict(q=q.data_ptr() + 8), dict(qt=9217), dict(oh=504), dict(ot=-8),
                    dict(sm=float("nan")), dict(sm=1e21), dict(out=None), dict(work=None), dict(bytes=need - 1),
                    dict(work=work.data_ptr() + 8), dict(lse=at + 2)]:
            assert call(**bad) == INVALID, bad
        torch.cuda.synchronize()
        assert torch.all(out == 0.25) and c.pool.get_error() == 0
        assert call(n=0) == 0 and call(segs=0) == 0
        torch.cuda.synchronize()
        assert torch.all(out == 0.25)
        assert call() == 0 and call(groups=0, gs=None, gl=None) == 0
        for sizes in ((-1, 1, 1), (16385, 1, 1), (1, 4097, 1), (1, 1, 2049)):
            with pytest.raises(H.HisparseError):
                c.pool.prefix_workspace_bytes(*sizes)


@pytest.mark.parametrize("heads", [16, 32, 64])
def test_the_smallest_calls(heads):
    """One token alone, in a group, over one position; two tokens that share a page; empty groups; a workspace that is
    larger than needed."""
    with Shared(heads, [2], [64], [65, 70]) as s:
        q = make_q(s.rng, 2, heads, "bf16")
        work = torch.empty(c_bytes(s.c, 100), dtype=torch.uint8, device="cuda")
        for groups, lens in (([0], []), ([0, 1], [64]), ([0, 0, 0], [64, 64]), ([1, 1], [0])):
            out, lse = run(s.c, groups, lens, [1], [0, 1], [70], q[:1], work=work)
            check_chunk(s.c, [s.kv[1]], [0], [0, 1], [70], q[:1], SM, out, lse, "bf16")
            out, lse = run(s.c, groups, lens, [0], [0, 1], [1], q[:1], work=work)
            check_chunk(s.c, [s.kv[0]], [0], [0, 1], [1], q[:1], SM, out, lse, "bf16")
        for lens in ([64], [0], [70]):
            out, lse = run(s.c, [0, 2], lens, [0, 1], [0, 1, 2], [65, 70], q, work=work)
            assert s.c.pool.get_error() == 0
            check_chunk(s.c, s.kv, [0, 1], [0, 1, 2], [65, 70], q, SM, out, lse, "bf16")


def c_bytes(c, n):
    return c.pool.prefix_workspace_bytes(n, n, n)


def test_the_largest_call():
    """As many tokens and segments as a call takes, in as many groups: more limits than the plan keeps in shared
    memory, several rounds of everything."""
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    n, segs, groups = H.PREFIX_MAX_TOKENS, H.CHUNK_MAX_SEGMENTS, H.PREFIX_MAX_GROUPS
    with Cache(heads=16, n_layers=2, lpi=2, pages=(40, 3, 2), max_ctx=2560) as c:
        rng = np.random.default_rng(0)
        kv = []
        for r, m in enumerate((2560, 192, 128)):
            x = rng.standard_normal((m, 576))
            rows = CP.pack_rows(x[:, :512], x[:, 512:])
            c.put_rows(1, r, np.arange(m), rows)
            kv.append(CP.row_values(rows))
        # 2,000 single tokens behind 2,432 positions, pairs of short groups, one long segment behind them
        req = np.r_[np.zeros(2000, int), np.repeat(rng.integers(0, 3, (segs - 2002) // 2), 2), 0, 0]
        starts = np.r_[0, 2000, 2000 + 2 * np.arange(1, groups - 1)]
        starts = np.minimum(np.r_[starts, segs], segs)
        lens = np.r_[2432, rng.integers(0, 129, groups - 1)]
        news = np.r_[np.ones(segs - 1, int), n - segs + 1]
        start = np.r_[0, np.cumsum(news)]
        top = np.array([2560, 192, 128])
        limit = np.concatenate([rng.integers(0, top[r] + 1, m) for r, m in zip(req, news)])
        q = make_q(rng, n, 16, "bf16")
        out, lse = run(c, starts, lens, req, start, limit, q)
        assert c.pool.get_error() == 0
        some = set(rng.choice(n, 150, replace=False).tolist()) | {0, 1999, 2000, segs - 2, segs - 1, n - 1}
        check_chunk(c, kv, req, start, limit, q, SM, out, lse, "bf16", some)
