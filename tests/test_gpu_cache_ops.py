"""The cache operators of prefill and dense decode on the GPU, through the C ABI, against
plain 64-bit implementations: quantised append (bit for bit), read back (bit for bit) and
chunk attention (within bounds derived from its number formats in cache_plain.py)."""
import ctypes
import math

import numpy as np
import pytest

import cache_plain as CP
from oracle.formats import e4m3_to_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
INVALID, BAD_ID, HOST_MISSING, RANGE = 1, 7, 6, 11


def dt(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


class Cache:
    """A pool of n_layers layers whose requests hold `pages` logical pages each at shuffled pool
    pages; every byte of the cache starts as 0xFF (e4m3 NaN codes, NaN scales and rope)."""

    def __init__(self, heads=16, n_layers=3, lpi=2, pages=(40,), fmt=None, max_ctx=None, spare=3, seed=0, fill=255,
                 host_pages=8):
        from sparse_mla_kv_indexer_gb300 import hisparse as H
        if not torch.cuda.is_available():
            pytest.skip("no CUDA device")
        self.H, self.heads, self.n_layers, self.lpi = H, heads, n_layers, lpi
        self.fmt = H.IDX_FP8 if fmt is None else fmt
        total = sum(pages) + spare
        self.n_pages = total
        self.max_ctx = max_ctx or -(-max(pages) * 64 // 128) * 128
        cfg = H.PoolConfig(page_size=64, row_bytes=656, idx_dim=128, n_idx_heads=16, n_heads=heads, topk=128,
                           n_layers=n_layers, layers_per_indexer=lpi, num_pages=total, num_idx_pages=total,
                           max_requests=len(pages), max_ctx=self.max_ctx, max_q_per_req=1, hot_rows=64, max_tokens=2,
                           idx_format=self.fmt, host_pages=host_pages)
        n_groups = -(-n_layers // lpi)
        self.page_bytes = 8448 if self.fmt == H.IDX_FP8 else 8192
        self.kv = [torch.full((total * 64, 656), fill, dtype=torch.uint8, device="cuda") for _ in range(n_layers)]
        self.idx = [torch.full((total, self.page_bytes), 255, dtype=torch.uint8, device="cuda") for _ in range(n_groups)]
        self.host = torch.full((host_pages, n_layers, 64, 656), 255, dtype=torch.uint8).pin_memory()
        self.pool = H.Pool(cfg, self.kv, self.idx, self.host)
        perm = np.random.default_rng(seed).permutation(total)
        self.table, self.idx_table, at = [], [], 0
        for r, k in enumerate(pages):
            self.table.append(perm[at:at + k].copy())
            self.idx_table.append(perm[::-1][at:at + k].copy())
            at += k
            self.pool.set_pages(r, 0, block_table=list(self.table[r]), idx_pages=list(self.idx_table[r]))
        self.work = torch.empty(self.pool.chunk_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        self.pool.close()

    def rows_at(self, r, pos):
        pos = np.asarray(pos)
        return self.table[r][pos // 64] * 64 + pos % 64

    def put_rows(self, layer, r, pos, rows):
        ids = torch.from_numpy(self.rows_at(r, pos)).cuda()
        self.kv[layer][ids] = torch.from_numpy(np.ascontiguousarray(rows)).cuda()

    def get_rows(self, layer, r, pos):
        return self.kv[layer][torch.from_numpy(self.rows_at(r, pos)).cuda()].cpu().numpy()

    def get_keys(self, layer, r, pos):
        """Codes [n, 128] and scales [n] (None for int8)."""
        idx = self.idx[layer // self.lpi].cpu().numpy()
        pos = np.asarray(pos)
        pg, off = self.idx_table[r][pos // 64], pos % 64
        codes = idx[:, :8192].reshape(-1, 64, 128)[pg, off]
        if self.fmt == self.H.IDX_INT8:
            return codes, None
        return codes, np.ascontiguousarray(idx[:, 8192:]).view("<f4")[pg, off]


def values(rng, n, width, dtype, spread=1.0):
    """n rows of values exactly representable in dtype, as a device tensor and as fp32."""
    x = rng.standard_normal((n, width)) * np.exp(spread * rng.standard_normal((n, 1)))
    t = torch.from_numpy(x.astype(np.float32)).to(dt(dtype))
    return t.cuda(), t.float().numpy()


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


# ---- append and read ---------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [1, 7, 64, 301])
def test_append_writes_the_definition_bit_for_bit(dtype, fmt, n):
    rng = np.random.default_rng(n + 10 * fmt)
    with Cache(pages=(9, 6), fmt=fmt) as c:
        n0 = n - n // 3
        req = np.r_[np.zeros(n0), np.ones(n - n0)].astype(np.int32)
        pos = np.r_[rng.permutation(9 * 64)[:n0], 5 + np.arange(n - n0)].astype(np.int32)
        proj, pf = values(rng, n, 640, dtype)       # latent | rope | 64 unused columns
        keys, kf = values(rng, n, 128, dtype)
        if n > 2:
            proj[1, :128] = 0                        # a group of zeros
            proj[2, 128:256] = 0
            proj[2, 130] = 2.0 ** -24                # one subnormal fp16 value in its group
            pf = proj.float().cpu().numpy()
            keys[1] = 0
            kf = keys.float().cpu().numpy()
        before = [k.clone() for k in c.kv]
        c.pool.append_quantized(2, i32(req), i32(pos), proj[:, :512], proj[:, 512:576], keys, key_scale=0.03125)
        assert c.pool.get_error() == 0
        want = CP.pack_rows(pf[:, :512], pf[:, 512:576])
        for r, sel in ((0, slice(0, n0)), (1, slice(n0, n))):
            if pos[sel].size == 0:
                continue
            assert np.array_equal(c.get_rows(2, r, pos[sel]), want[sel])
            codes, scales = c.get_keys(2, r, pos[sel])
            if fmt == c.H.IDX_FP8:
                wc, ws = CP.quantise(kf[sel])
                assert np.array_equal(codes, wc) and np.array_equal(scales, ws[:, 0])
            else:
                wk = np.clip(np.rint(kf[sel].astype(np.float64) / 0.03125), -127, 127).astype(np.int8)
                assert np.array_equal(codes.view(np.int8), wk)
        assert torch.equal(c.kv[0], before[0]) and torch.equal(c.kv[1], before[1])
        touched = torch.zeros(c.n_pages * 64, dtype=torch.bool)
        for r, sel in ((0, slice(0, n0)), (1, slice(n0, n))):
            touched[torch.from_numpy(c.rows_at(r, pos[sel]).astype(np.int64))] = True
        assert torch.equal(c.kv[2].cpu()[~touched], before[2].cpu()[~touched])


def test_append_parts_padding_duplicates_and_bad_ids():
    rng = np.random.default_rng(3)
    with Cache(pages=(4, 4)) as c:
        c.pool.set_pages(1, 2, block_table=[-1])      # page 2 of request 1 is a placeholder
        lat, lf = values(rng, 6, 512, "bf16")
        rope, rf = values(rng, 6, 64, "bf16")
        keys, kf = values(rng, 6, 128, "bf16")
        # token 1 is padding; tokens 2 and 3 give one position twice: the later one stays;
        # token 4's row has no page but its key has; token 5 is in order
        req, pos = i32([0, -1, 0, 0, 1, 1]), i32([7, 9, 70, 70, 130, 3])
        c.pool.append_quantized(0, req, pos, lat, rope, keys)
        assert c.pool.get_error() == BAD_ID
        want = CP.pack_rows(lf, rf)
        assert np.array_equal(c.get_rows(0, 0, [7, 70]), want[[0, 3]])
        assert np.array_equal(c.get_rows(0, 1, [3]), want[[5]])
        assert np.all(c.get_rows(0, 0, [9]) == 255)
        wc, ws = CP.quantise(kf)
        codes, scales = c.get_keys(0, 1, [130, 3])
        assert np.array_equal(codes, wc[[4, 5]]) and np.array_equal(scales, ws[[4, 5], 0])
        # rows alone, then keys alone: the other part stays
        snap = [c.kv[1].clone(), c.idx[0].clone()]
        c.pool.append_quantized(1, req[:1], pos[:1], lat[:1], rope[:1])
        assert torch.equal(c.idx[0], snap[1]) and np.array_equal(c.get_rows(1, 0, [7]), want[:1])
        snap = [c.kv[1].clone(), c.idx[1].clone()]
        c.pool.append_quantized(2, req[:1], pos[:1], keys=keys[:1])
        assert torch.equal(c.kv[1], snap[0]) and np.array_equal(c.get_keys(2, 0, [7])[0], wc[:1])
        assert c.pool.get_error() == 0
        snap = [k.clone() for k in c.kv + c.idx]
        for r, p in [(2, 0), (-2, 0), (0, c.max_ctx), (0, -1)]:
            c.pool.append_quantized(0, i32([r]), i32([p]), lat[:1], rope[:1], keys[:1])
            assert c.pool.get_error() == BAD_ID, (r, p)
        assert all(torch.equal(a, b) for a, b in zip(snap, c.kv + c.idx))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_of_values_that_are_not_finite(dtype):
    rng = np.random.default_rng(4)
    with Cache(pages=(2,)) as c:
        lat, lf = values(rng, 2, 512, dtype)
        rope, rf = values(rng, 2, 64, dtype)
        lat[0, 5], lat[0, 300], rope[0, 3] = float("nan"), float("-inf"), float("nan")
        rope[0, 4] = float("inf")
        c.pool.append_quantized(0, i32([0, 0]), i32([0, 1]), lat, rope)
        assert c.pool.get_error() == RANGE
        lf, rf = lf.copy(), rf.copy()
        lf[0, 5], lf[0, 300], rf[0, 3], rf[0, 4] = 0, 0, 0, 0
        want = CP.pack_rows(lf, rf)
        want[0, 300] = 0xFE                            # -448
        want[0, 528 + 8:528 + 10] = [0x7F, 0x7F]       # the largest finite bf16
        assert np.array_equal(c.get_rows(0, 0, [0, 1]), want)


@pytest.mark.parametrize("magnitude", [1e-38, 1e-30, 1e30])
def test_append_of_tiny_and_huge_values(magnitude):
    rng = np.random.default_rng(5)
    with Cache(pages=(2,)) as c:
        lat = torch.from_numpy((rng.standard_normal((3, 512)) * magnitude).astype(np.float32)).cuda()
        rope = torch.zeros(3, 64, device="cuda")
        c.pool.append_quantized(0, i32([0, 0, 0]), i32([0, 1, 64]), lat, rope)
        assert c.pool.get_error() == 0
        assert np.array_equal(c.get_rows(0, 0, [0, 1, 64]), CP.pack_rows(lat.cpu().numpy(), rope.cpu().numpy()))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [1, 9, 200])
def test_read_returns_code_times_scale_rounded_once(dtype, fmt, n):
    rng = np.random.default_rng(n)
    with Cache(pages=(6,), fmt=fmt) as c:
        rows = CP.pack_rows(rng.standard_normal((384, 512)), rng.standard_normal((384, 64)))
        c.put_rows(1, 0, np.arange(384), rows)
        codes = rng.integers(0, 127, (c.n_pages, c.page_bytes), dtype=np.uint8)
        if fmt == c.H.IDX_FP8:
            codes[:, 8192:] = np.abs(rng.standard_normal((c.n_pages, 64))).astype("<f4").view(np.uint8).reshape(c.n_pages, -1)
        c.idx[0].copy_(torch.from_numpy(codes))
        pos = rng.integers(0, 384, n)
        if n > 4:
            pos[1] = pos[3]                            # the same position twice
        req = np.zeros(n, np.int32)
        if n > 4:
            req[4] = -1
        wide = torch.full((n, 720), 7.0, dtype=dt(dtype), device="cuda")
        lat, rope, keys = wide[:, 8:520], wide[:, 520:584], wide[:, 584:712]
        c.pool.read_rows(1, i32(req), i32(pos), lat, rope, keys, key_scale=0.125)
        assert c.pool.get_error() == 0
        v = CP.row_values(rows[pos])
        kc, ks = c.get_keys(1, 0, pos)
        kv = e4m3_to_f64(kc) * ks[:, None].astype(np.float64) if fmt == c.H.IDX_FP8 else kc.view(np.int8) * 0.125
        want = torch.full((n, 720), 7.0, dtype=dt(dtype))
        live = torch.from_numpy(req >= 0)
        # the product of a 4-bit code and an fp32 scale is rounded to fp32, then to the output type
        want[live, 8:584] = torch.from_numpy(v.astype(np.float32)).to(dt(dtype))[live]
        want[live, 584:712] = torch.from_numpy(kv.astype(np.float32)).to(dt(dtype))[live]
        assert torch.equal(wide.cpu(), want)
        one = torch.full((n, 64), 7.0, dtype=dt(dtype), device="cuda")
        c.pool.read_rows(1, i32(req), i32(pos), rope=one)
        assert torch.equal(one.cpu()[live], want[live, 520:584])


def test_read_from_host_copies_and_missing_pages():
    rng = np.random.default_rng(8)
    with Cache(pages=(4,)) as c:
        rows = CP.pack_rows(rng.standard_normal((256, 512)), rng.standard_normal((256, 64)))
        c.put_rows(2, 0, np.arange(256), rows)
        c.host[5, 2] = torch.from_numpy(rows[64:128])
        c.pool.set_pages(0, 1, block_table=[-1, -1], host_pages=[5, -1])
        pos = [63, 64, 100, 127, 128, 192]
        lat = torch.full((6, 512), 3.0, device="cuda")
        c.pool.read_rows(2, i32([0] * 6), i32(pos), lat)
        assert c.pool.get_error() == HOST_MISSING
        want = CP.row_values(rows[pos])[:, :512].astype(np.float32)
        want[4] = 3.0
        assert np.array_equal(lat.cpu().numpy(), want)


def test_append_then_read_round_trip_and_a_fork_between_requests():
    """Rows read from one request and appended to another quantise to the same rows: amax is a
    code of +-448 times the scale, so scale and codes come back."""
    rng = np.random.default_rng(9)
    with Cache(pages=(3, 3)) as c:
        lat, _ = values(rng, 150, 512, "fp32")
        rope, _ = values(rng, 150, 64, "bf16")
        pos = i32(np.arange(150))
        c.pool.append_quantized(0, i32(np.zeros(150)), pos, lat, rope.float())
        out, ro = torch.empty_like(lat), torch.empty(150, 64, device="cuda")
        c.pool.read_rows(0, i32(np.zeros(150)), pos, out, ro)
        c.pool.append_quantized(0, i32(np.ones(150)), pos, out, ro)
        assert c.pool.get_error() == 0
        a, b = c.get_rows(0, 0, np.arange(150)), c.get_rows(0, 1, np.arange(150))
        assert np.array_equal(CP.row_values(a), CP.row_values(b))


@pytest.mark.parametrize("n", [9729, 20011, 170001])
def test_a_large_call_equals_its_pieces(n):
    """Warps that take runs of several tokens, up to the longest run, the last one cut short:
    padding and positions given twice at odd places, two thirds of the padding in one stretch."""
    rng = np.random.default_rng(n)
    pages = -(-n // 64) + 1
    with Cache(n_layers=1, lpi=1, pages=(pages, pages)) as c:
        lat, _ = values(rng, n, 512, "bf16")
        rope, _ = values(rng, n, 64, "bf16")
        keys, _ = values(rng, n, 128, "bf16")
        pos = rng.permutation(pages * 64)[:n]
        twice = rng.choice(np.arange(1, n), n // 20, replace=False)
        twice = np.r_[twice, [31, 32, 33, 64, n - 1]]
        for j in np.sort(twice):
            pos[j] = pos[j - 1]
        req = np.zeros(n, np.int32)
        req[rng.choice(n, n // 50, replace=False)] = -1
        req[n // 3:n // 3 + n // 25] = -1
        live = np.flatnonzero(req >= 0)                # a position again behind padding is not adjacent: not allowed
        again = np.flatnonzero((pos[live[1:]] == pos[live[:-1]]) & (np.diff(live) > 1)) + 1
        req[live[again]] = -1
        c.pool.append_quantized(0, i32(req), i32(pos), lat, rope, keys)
        cut = [0]
        while cut[-1] < n:                              # never between the two of one position
            e = min(cut[-1] + 4000, n)
            while e < n and pos[e] == pos[e - 1]:
                e += 1
            cut.append(e)
        for a, b in zip(cut, cut[1:]):
            c.pool.append_quantized(0, i32(np.where(req[a:b] < 0, -1, 1)), i32(pos[a:b]), lat[a:b], rope[a:b], keys[a:b])
        assert c.pool.get_error() == 0
        every = np.arange(pages * 64)
        assert np.array_equal(c.get_rows(0, 0, every), c.get_rows(0, 1, every))
        for a, b in zip(c.get_keys(0, 0, every), c.get_keys(0, 1, every)):
            assert np.array_equal(a.view(np.uint8), b.view(np.uint8))
        got, want = (torch.full((n, 704), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        c.pool.read_rows(0, i32(req), i32(pos), got[:, :512], got[:, 512:576], got[:, 576:])
        for a in range(0, n, 4000):
            w = want[a:a + 4000]
            c.pool.read_rows(0, i32(req[a:a + 4000]), i32(pos[a:a + 4000]), w[:, :512], w[:, 512:576], w[:, 576:])
        assert c.pool.get_error() == 0
        assert torch.equal(got, want) and not torch.isnan(got.float()).any()


def test_the_most_tokens_of_a_call():
    """Values whose offsets pass 2^31 elements."""
    rng = np.random.default_rng(11)
    with Cache(n_layers=1, lpi=1, pages=(8,)) as c:
        n, H = c.H.CACHE_MAX_TOKENS, c.H
        some, _ = values(rng, 500, 128, "fp16")
        keys = torch.zeros(n, 128, dtype=torch.float16, device="cuda")
        at = torch.from_numpy(np.sort(rng.choice(n - 1, 499, replace=False))).cuda()
        at = torch.cat([at, torch.tensor([n - 1], device="cuda")])
        req, pos = torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        req[at], pos[at], keys[at] = 0, torch.arange(500, dtype=torch.int32, device="cuda"), some
        c.pool.append_quantized(0, req, pos, keys=keys)
        assert c.pool.get_error() == 0
        codes, scales = c.get_keys(0, 0, np.arange(500))
        wc, ws = CP.quantise(some.float().cpu().numpy())
        assert np.array_equal(codes, wc) and np.array_equal(scales, ws[:, 0])
        table = torch.empty(500, 128, dtype=torch.float16, device="cuda")
        every = i32(np.arange(500))
        c.pool.read_rows(0, i32(np.zeros(500)), every, keys=table)
        pos = torch.randint(0, 500, (n,), dtype=torch.int32, device="cuda")
        keys.fill_(9.0)
        c.pool.read_rows(0, torch.zeros_like(pos), pos, keys=keys)
        assert c.pool.get_error() == 0
        for a in range(0, n, 1 << 21):
            assert torch.equal(keys[a:a + (1 << 21)], table[pos[a:a + (1 << 21)].long()]), a
        with pytest.raises(H.HisparseError):
            more = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
            c.pool.read_rows(0, more, more, keys=torch.empty(n + 1, 128, dtype=torch.float16, device="cuda"))


# ---- chunk attention ---------------------------------------------------------------


def fill(c, rng, layer, lengths, sink=False):
    """Random rows at positions [0, lengths[r]) of every request; returns their values."""
    kv = []
    for r, n in enumerate(lengths):
        x = rng.standard_normal((n, 576)) * np.exp(0.3 * rng.standard_normal((n, 1)))
        if sink and n:
            x[0] *= 6.0
        rows = CP.pack_rows(x[:, :512], x[:, 512:]) if n else np.zeros((0, 656), np.uint8)
        if n:
            c.put_rows(layer, r, np.arange(n), rows)
        kv.append(CP.row_values(rows))
    return kv


def run_chunk(c, layer, seg_req, seg_start, limit, q, sm_scale, n_out=None, lse=True, out=None, stream=None):
    n = q.shape[0]
    out = torch.full((n, c.heads, 512), 0.25, dtype=q.dtype, device="cuda") if out is None else out
    l = torch.full((n, c.heads), 0.25, device="cuda") if lse else None
    c.pool.chunk_attention(layer, i32(seg_req), i32(seg_start), i32(limit), q, sm_scale, out, c.work, lse=l, stream=stream)
    return out, l


def check_chunk(c, kv, seg_req, seg_start, limit, q, sm_scale, out, lse, dtype, tokens=None):
    """Every token of every segment within the derived bounds; tokens outside untouched."""
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    qf = q.float().cpu().numpy().astype(np.float64)
    inside = np.zeros(q.shape[0], bool)
    for i, r in enumerate(seg_req):
        for j in range(seg_start[i], seg_start[i + 1]):
            inside[j] = True
            if tokens is not None and j not in tokens:
                continue
            k = kv[r][:limit[j]]
            wo, wl, a, s = CP.attend(qf[j], k, sm_scale)
            if limit[j] == 0:
                assert np.all(o[j] == 0) and np.all(np.isneginf(l[j])), j
                continue
            err = np.abs(o[j] - wo)
            b = CP.out_bound(wo, a, s, HALF_STEP[dtype], k.shape[0])
            assert np.all(err <= b), (i, j, int(limit[j]), float((err / b).max()), float(err.max()))
            el = np.abs(l[j] - wl)
            assert np.all(el <= CP.lse_bound(wl, s)), (i, j, float(el.max()))
    assert np.all(o[~inside] == 0.25) and np.all(l[~inside] == 0.25)


def make_q(rng, n, heads, dtype, size=1.5):
    return torch.from_numpy((size * rng.standard_normal((n, heads, 576))).astype(np.float32)).to(dt(dtype)).cuda()


@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_chunk_ragged_segments(heads, dtype):
    """Segments of 1 to 70 tokens over contexts of 1 to 2,500 rows, an empty segment, a token
    that sees nothing, limits out of order, tokens before, between and behind the segments."""
    rng = np.random.default_rng(heads)
    lengths = [1, 63, 64, 65, 2500, 300, 129]
    with Cache(heads=heads, pages=[max(1, -(-n // 64)) for n in lengths]) as c:
        kv = fill(c, rng, 1, lengths, sink=True)
        news = [1, 2, 64, 5, 3, 70, 0, 9]
        seg_req = [0, 1, 2, 3, 4, 5, 0, 6]
        start = np.r_[2, 2 + np.cumsum(news)]          # two tokens before the first segment
        n = int(start[-1]) + 4                         # four behind the last
        limit = np.full(n, 5)
        for i, r in enumerate(seg_req):
            lo, hi = start[i], start[i + 1]
            limit[lo:hi] = np.arange(lengths[r] - news[i] + 1, lengths[r] + 1)
        a, b = start[5], start[6]
        limit[a:b] = rng.permutation(limit[a:b])
        limit[a + 7] = 0
        limit[start[7] + 8] = 0
        q = make_q(rng, n, heads, dtype)
        sm = 1 / math.sqrt(576)
        out, lse = run_chunk(c, 1, seg_req, start, limit, q, sm)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, seg_req, start, limit, q, sm, out, lse, dtype)
        again, lse2 = run_chunk(c, 1, seg_req, start, limit, q, sm)
        assert torch.equal(out, again) and torch.equal(lse, lse2)     # the same call, the same bits


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 127, 128, 129, 640, 5000])
def test_chunk_single_token(heads, length):
    rng = np.random.default_rng(length)
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(-(-length // 64),)) as c:
        kv = fill(c, rng, 0, [length])
        q = make_q(rng, 1, heads, "bf16")
        out, lse = run_chunk(c, 0, [0], [0, 1], [length], q, 1 / 24)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, [0], [0, 1], [length], q, 1 / 24, out, lse, "bf16")


@pytest.mark.parametrize("heads,new", [(64, 200), (16, 777), (32, 131)])
def test_chunk_prompt_from_its_first_token(heads, new):
    rng = np.random.default_rng(new)
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(-(-new // 64),)) as c:
        kv = fill(c, rng, 0, [new], sink=True)
        q = make_q(rng, new, heads, "bf16")
        limit = np.arange(1, new + 1)
        out, lse = run_chunk(c, 0, [0], [0, new], limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        some = set(range(0, new, 13)) | set(range(8)) | {new - 1}
        check_chunk(c, kv, [0], [0, new], limit, q, 1 / 24, out, lse, "bf16", some)


def test_chunk_more_blocks_than_threads():
    """A prompt of 1,450 blocks, planned in three rounds of the CTA's threads, behind 700 single
    tokens and with empty segments between."""
    rng = np.random.default_rng(13)
    with Cache(heads=64, n_layers=1, lpi=1, pages=(46, 4)) as c:
        kv = fill(c, rng, 0, [2900, 256])
        seg_req = [1, 1] * 700 + [0, 1]
        start = np.r_[0, np.repeat(np.arange(1, 701), 2), 700 + 2900, 700 + 2900]
        limit = np.r_[rng.integers(0, 257, 700), np.arange(1, 2901)]
        q = make_q(rng, 3600, 64, "bf16")
        out, lse = run_chunk(c, 0, seg_req, start, limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        some = set(range(0, 700, 60)) | set(range(700, 3600, 290)) | {3599}
        check_chunk(c, kv, seg_req, start, limit, q, 1 / 24, out, lse, "bf16", some)


def test_chunk_most_segments_and_tokens_of_a_call():
    """4,096 segments of 16 tokens, 65,536 tokens in all, over short contexts."""
    rng = np.random.default_rng(14)
    with Cache(heads=16, n_layers=1, lpi=1, pages=(2, 1)) as c:
        kv = fill(c, rng, 0, [100, 64])
        n, segs = 65536, 4096
        q = make_q(rng, 64, 16, "bf16").repeat(n // 64, 1, 1)
        limit = np.tile(np.r_[np.arange(85, 101), np.arange(49, 65)], n // 32)
        seg_req = np.tile([0, 1], segs // 2)
        start = np.arange(segs + 1) * 16
        out, lse = run_chunk(c, 0, seg_req, start, limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        few = [slice(0, 64), slice(n // 2, n // 2 + 64), slice(n - 64, n)]
        for s in few:      # the same inputs: the same bits, wherever a pair's range was cut or not
            o, l = out[s].float().cpu().numpy(), lse[s].cpu().numpy()
            for j in range(0, 64, 5):
                wo, wl, a, sz = CP.attend(q[j].float().cpu().numpy().astype(np.float64),
                                          kv[int(seg_req[j // 16])][:limit[j]], 1 / 24)
                assert np.all(np.abs(o[j] - wo) <= CP.out_bound(wo, a, sz, HALF_STEP["bf16"], limit[j]))
                assert np.all(np.abs(l[j] - wl) <= CP.lse_bound(wl, sz))
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


def test_two_calls_at_once_on_two_streams():
    """Two pools' caches, two streams, a workspace each: the calls overlap as they like."""
    rng = np.random.default_rng(15)
    with Cache(heads=64, n_layers=1, lpi=1, pages=(40,), seed=1) as c, Cache(heads=16, n_layers=1, lpi=1, pages=(40,)) as d:
        s = [torch.cuda.Stream(), torch.cuda.Stream()]
        sides = []
        for x in (c, d):
            kv = fill(x, rng, 0, [2500])
            q = make_q(rng, 40, x.heads, "bf16")
            limit = np.arange(2461, 2501)
            args = (i32([0]), i32([0, 40]), i32(limit))
            sides.append((kv, q, limit, args, [torch.full((40, x.heads, 512), 0.25, dtype=torch.bfloat16, device="cuda") for _ in range(4)],
                          [torch.full((40, x.heads), 0.25, device="cuda") for _ in range(4)]))
        torch.cuda.synchronize()
        for rep in range(4):
            for x, st, (kv, q, limit, args, outs, lses) in zip((c, d), s, sides):
                x.pool.chunk_attention(0, *args, q, 1 / 24, outs[rep], x.work, lse=lses[rep], stream=st)
        torch.cuda.synchronize()
        for x, (kv, q, limit, args, outs, lses) in zip((c, d), sides):
            assert x.pool.get_error() == 0
            check_chunk(x, kv, [0], [0, 40], limit, q, 1 / 24, outs[0], lses[0], "bf16", {0, 17, 39})
            for o, l in zip(outs[1:], lses[1:]):
                assert torch.equal(o, outs[0]) and torch.equal(l, lses[0])


def test_chunk_many_single_token_segments():
    """More segments than thread-block pairs on the GPU, lengths from nothing to 700 rows."""
    rng = np.random.default_rng(12)
    n = 333
    lengths = rng.integers(1, 700, n)
    with Cache(heads=64, n_layers=1, lpi=1, pages=[-(-int(x) // 64) for x in lengths]) as c:
        kv = fill(c, rng, 0, lengths)
        limit = lengths.copy()
        limit[::50] = 0
        q = make_q(rng, n, 64, "bf16")
        out, lse = run_chunk(c, 0, np.arange(n), np.arange(n + 1), limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, np.arange(n), np.arange(n + 1), limit, q, 1 / 24, out, lse, "bf16", set(range(0, n, 10)))


@pytest.mark.parametrize("sm_scale", [0.0, 0.5, -0.1])
def test_chunk_scales(sm_scale):
    """No scale (a plain mean), a sharp softmax whose maximum moves late, a negative scale."""
    rng = np.random.default_rng(20)
    with Cache(heads=16, n_layers=1, lpi=1, pages=(15,)) as c:
        kv = fill(c, rng, 0, [900])
        q = make_q(rng, 9, 16, "bf16")
        q[3] = torch.from_numpy(kv[0][899]).to(torch.bfloat16).cuda()      # the last row wins for every head of token 3
        limit = np.arange(892, 901)
        out, lse = run_chunk(c, 0, [0], [0, 9], limit, q, sm_scale)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, [0], [0, 9], limit, q, sm_scale, out, lse, "bf16")


def test_chunk_dominant_row_and_a_long_faint_tail():
    """One row takes about half of the weight and the other 6,399 share the rest: probabilities
    of 2^-14 and below of the largest keep their precision."""
    rng = np.random.default_rng(21)
    with Cache(heads=16, n_layers=1, lpi=1, pages=(100,)) as c:
        n = 6400
        x = np.zeros((n, 576))
        x[:, 0] = 1.0                                  # every row but the first scores 0 on q = e_1
        x[:, 2] = 1.25                                 # and carries a value that adds up
        x[0] = 0
        x[0, 1] = 1.0
        rows = CP.pack_rows(x[:, :512], x[:, 512:])
        c.put_rows(0, 0, np.arange(n), rows)
        kv = [CP.row_values(rows)]
        q = torch.zeros(3, 16, 576, dtype=torch.bfloat16, device="cuda")
        q[:, :, 1] = torch.tensor([8.75, 10.5, 13.0], device="cuda")[:, None].to(torch.bfloat16)
        limit = [n, n, n]
        out, lse = run_chunk(c, 0, [0], [0, 3], limit, q, 1.0)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, [0], [0, 3], limit, q, 1.0, out, lse, "bf16")


@pytest.mark.parametrize("heads", [16, 64])
def test_chunk_up_to_the_longest_context(heads):
    """Limits of max_ctx itself, for one token and for many; one more is refused by the kernel."""
    rng = np.random.default_rng(30)
    with Cache(heads=heads, n_layers=1, lpi=1, pages=(4, 4), max_ctx=256) as c:
        kv = fill(c, rng, 0, [256, 256])
        q = make_q(rng, 21, heads, "bf16")
        limit = np.r_[np.full(20, 256), 256]
        out, lse = run_chunk(c, 0, [0, 1], [0, 20, 21], limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, [0, 1], [0, 20, 21], limit, q, 1 / 24, out, lse, "bf16")
        limit[3] = 257
        out, lse = run_chunk(c, 0, [0, 1], [0, 20, 21], limit, q, 1 / 24)
        assert c.pool.get_error() == BAD_ID
        assert torch.all(out[3] == 0) and torch.all(torch.isneginf(lse[3]))
        check_chunk(c, kv, [0, 1], [0, 20, 21], limit, q, 1 / 24, out, lse, "bf16", set(range(21)) - {3})


def test_chunk_strides_and_no_lse():
    rng = np.random.default_rng(22)
    with Cache(heads=32, n_layers=1, lpi=1, pages=(5,)) as c:
        kv = fill(c, rng, 0, [300])
        n = 11
        base = make_q(rng, 32, n, "bf16")              # [head, token, 576]
        wide = torch.zeros(32, n, 584, dtype=torch.bfloat16, device="cuda")
        wide[:, :, 8:] = base
        q = wide[:, :, 8:].transpose(0, 1)             # a view: token stride 584, head stride n * 584
        flat = torch.full((32, n, 520), 0.25, dtype=torch.bfloat16, device="cuda")
        out = flat[:, :, :512].transpose(0, 1)
        limit = np.arange(290, 301)
        run_chunk(c, 0, [0], [0, n], limit, q, 1 / 24, out=out, lse=False)
        ref, lse = run_chunk(c, 0, [0], [0, n], limit, q.contiguous(), 1 / 24)
        assert c.pool.get_error() == 0
        assert torch.equal(out.contiguous(), ref) and torch.all(flat[:, :, 512:] == 0.25)
        check_chunk(c, kv, [0], [0, n], limit, q, 1 / 24, ref, lse, "bf16")
        one = make_q(rng, 1, 1, "bf16").expand(n, 32, 576)         # one query for every token and head
        a, _ = run_chunk(c, 0, [0], [0, n], limit, one, 1 / 24)
        b, _ = run_chunk(c, 0, [0], [0, n], limit, one.contiguous(), 1 / 24)
        assert torch.equal(a, b)


def test_chunk_ignores_what_no_token_sees():
    """Rows at and beyond every limit hold NaN codes, scales and rope (0xFF), and a page whose
    rows nobody sees is a placeholder without a host copy."""
    rng = np.random.default_rng(23)
    with Cache(heads=64, n_layers=1, lpi=1, pages=(8,)) as c:
        kv = fill(c, rng, 0, [101])
        c.pool.set_pages(0, 2, block_table=[-1] * 6)
        q = make_q(rng, 3, 64, "bf16")
        limit = [99, 100, 101]
        out, lse = run_chunk(c, 0, [0], [0, 3], limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, [0], [0, 3], limit, q, 1 / 24, out, lse, "bf16")


def test_chunk_values_out_of_range_are_reported_and_not_seen():
    rng = np.random.default_rng(24)
    with Cache(heads=16, n_layers=1, lpi=1, pages=(4,)) as c:
        n = 200
        rows = CP.pack_rows(rng.standard_normal((n, 512)), rng.standard_normal((n, 64)))
        good = rows.copy()
        rows[10, 37] = 0x7F                            # a NaN code
        rows[20, 516:520] = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)
        rows[30, 520:524] = np.frombuffer(np.float32(200.0).tobytes(), np.uint8)
        rows[40, 528:530] = [0x80, 0x7F]               # rope infinity
        c.put_rows(0, 0, np.arange(n), rows)
        q = make_q(rng, 4, 16, "bf16")
        limit = np.arange(197, 201)
        out, lse = run_chunk(c, 0, [0], [0, 4], limit, q, 1 / 24)
        assert c.pool.get_error() == RANGE
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
        rows = good.copy()
        rows[50, 530:532] = [0x80, 0xFF]               # minus infinity at a rope value that every query
        q1 = q.clone()                                 # has positive: its score is -inf everywhere
        q1[:, :, 513] = 1.0
        c.put_rows(0, 0, np.arange(n), rows)
        out, lse = run_chunk(c, 0, [0], [0, 4], limit, q1, 1 / 24)
        assert c.pool.get_error() == RANGE
        kv = CP.row_values(good)
        rest = np.r_[0:50, 51:n]                       # the row counts as not seen
        check_chunk(c, [kv[rest]], [0], [0, 4], limit - 1, q1, 1 / 24, out, lse, "bf16")
        c.put_rows(0, 0, np.arange(n), good)
        q[2, 3, 100] = 70000.0                         # beyond fp16
        out, lse = run_chunk(c, 0, [0], [0, 4], limit, q, 1 / 24)
        assert c.pool.get_error() == RANGE
        assert torch.all(out[2, 3] == 0) and lse[2, 3] == float("-inf")     # that query row sees nothing
        q0 = q.clone()
        q0[2, 3, 100] = 0
        keep = [0, 1, 3]
        check_chunk(c, [CP.row_values(good)], [0], [0, 4], limit, q0, 1 / 24, out, lse, "bf16", set(keep))


@pytest.mark.parametrize("sm_scale", [1.0, -1.0, 64.0])
def test_chunk_scores_too_large_are_reported_and_not_seen(sm_scale):
    """A row whose scores are 2.5e8 or more for one query and minus that for another: the first
    does not see it, for the second its weight is 0 by the formula; a query that has no score
    in range sees nothing."""
    rng = np.random.default_rng(26)
    with Cache(heads=16, n_layers=1, lpi=1, pages=(4,)) as c:
        n = 200
        x = np.zeros((n, 576))
        x[:, 1:512] = rng.standard_normal((n, 511)) / 32
        rows = CP.pack_rows(x[:, :512], x[:, 512:])
        rows[70:71] = CP.pack_rows(np.where(np.arange(512) == 0, 4096.0, x[70:71, :512]), x[70:71, 512:])
        c.put_rows(0, 0, np.arange(n), rows)
        q = torch.zeros(4, 16, 576, dtype=torch.bfloat16, device="cuda")
        q[:, :, 1:] = make_q(rng, 4, 16, "bf16")[:, :, 1:] / abs(sm_scale)
        limit = np.array([200, 200, 71, 70])
        sign = 1.0 if sm_scale > 0 else -1.0
        q[0, :, 0] = 60000.0 * sign                    # z = 2.5e8 |sm_scale|
        q[1, :, 0] = -60000.0 * sign
        out, lse = run_chunk(c, 0, [0], [0, 4], limit, q, sm_scale)
        assert c.pool.get_error() == RANGE             # token 0's
        without = CP.row_values(rows)[np.r_[0:70, 71:n]]
        check_chunk(c, [without], [0], [0, 4], np.array([199, 199, 70, 70]), q, sm_scale, out, lse, "bf16", {0, 1, 3})
        check_chunk(c, [CP.row_values(rows)], [0], [0, 4], limit, q, sm_scale, out, lse, "bf16", {1, 2, 3})
        out, lse = run_chunk(c, 0, [0], [0, 3], limit[1:], q[1:], sm_scale)
        assert c.pool.get_error() == 0                 # a low score beside others is no error
        c.put_rows(0, 0, np.arange(n), np.repeat(rows[70:71], n, axis=0))
        out, lse = run_chunk(c, 0, [0], [0, 2], limit[:2], q[:2], sm_scale)
        assert c.pool.get_error() == RANGE
        assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
        out, lse = run_chunk(c, 0, [0], [0, 1], limit[1:2], q[1:2], sm_scale)
        assert c.pool.get_error() == RANGE             # none in range from below
        assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("more", [0, 60])
def test_chunk_bad_ids_leave_the_other_segments_right(more):
    """With `more` empty segments behind, the call is planned by the whole CTA instead of a warp."""
    rng = np.random.default_rng(25)
    with Cache(heads=16, n_layers=1, lpi=1, pages=(3, 3)) as c:
        kv = fill(c, rng, 0, [150, 150])
        q = make_q(rng, 8, 16, "bf16")

        def run(seg_req, start, limit):
            return run_chunk(c, 0, list(seg_req) + [0] * more, list(start) + [start[-1]] * more, limit, q, 1 / 24)
        for seg_req, start, limit in [([0, 9, 1], [0, 2, 5, 8], [100] * 8), ([0, -1, 1], [0, 2, 5, 8], [100] * 8),
                                      ([0, 0, 1], [0, 2, 5, 8], [100, 100, c.max_ctx + 1, -3, 1 << 30, 100, 100, 100])]:
            out, lse = run(seg_req, start, limit)
            assert c.pool.get_error() == BAD_ID
            check_chunk(c, kv, [0, 0, 1], [0, 2, 5, 8], limit, q, 1 / 24, out, lse, "bf16", {0, 1, 5, 6, 7})
            assert torch.all(out[2:5] == 0) and torch.all(lse[2:5] == float("-inf"))
        # starts out of order or range: clamped, reported
        for start in ([0, 6, 3, 8], [0, 2, 5, 9], [-4, 2, 5, 8]):
            out, lse = run([0, 0, 1], start, [100] * 8)
            assert c.pool.get_error() == BAD_ID


def test_chunk_reads_host_copies_and_reports_missing_pages():
    rng = np.random.default_rng(26)
    with Cache(heads=16, n_layers=2, lpi=1, pages=(5,)) as c:
        kv = fill(c, rng, 1, [300])
        for page, host in ((1, 3), (3, 6)):
            c.host[host, 1] = torch.from_numpy(c.get_rows(1, 0, np.arange(64 * page, 64 * page + 64)))
            c.put_rows(1, 0, np.arange(64 * page, 64 * page + 64), np.full((64, 656), 255, np.uint8))
            c.pool.set_pages(0, page, block_table=[-1], host_pages=[host])
        q = make_q(rng, 6, 16, "bf16")
        limit = np.arange(295, 301)
        out, lse = run_chunk(c, 1, [0], [0, 6], limit, q, 1 / 24)
        assert c.pool.get_error() == 0
        check_chunk(c, kv, [0], [0, 6], limit, q, 1 / 24, out, lse, "bf16")
        c.pool.set_pages(0, 2, block_table=[-1])       # neither resident nor on the host: not seen
        out, lse = run_chunk(c, 1, [0], [0, 6], limit, q, 1 / 24)
        assert c.pool.get_error() == HOST_MISSING
        rest = np.r_[0:128, 192:300]
        check_chunk(c, [kv[0][rest]], [0], [0, 6], limit - 64, q, 1 / 24, out, lse, "bf16")


def test_chunk_long_context_and_offsets_past_32_bits():
    """A token over 200,003 rows, whose pages lie at both ends of a 4.5 GB cache."""
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n, heads = 200003, 64
    pages, total = -(-n // 64), 108000                 # 108,000 pages of 41,984 bytes
    gen = torch.Generator("cuda").manual_seed(1)
    kv = torch.zeros(total * 64, 656, dtype=torch.uint8, device="cuda")
    table = torch.cat([torch.arange(pages // 2), torch.arange(total - (pages - pages // 2), total)]).cuda()
    ids = (table[:, None] * 64 + torch.arange(64, device="cuda")).flatten()[:n]
    codes = torch.randint(0, 127, (n, 512), generator=gen, device="cuda", dtype=torch.uint8) ^ \
        (torch.randint(0, 2, (n, 512), generator=gen, device="cuda", dtype=torch.uint8) << 7)
    scale = (0.002 + 0.002 * torch.rand(n, 4, generator=gen, device="cuda"))
    rope = torch.randn(n, 64, generator=gen, device="cuda").bfloat16()
    kv[ids] = torch.cat([codes, scale.view(torch.uint8), rope.view(torch.uint8)], 1)
    cfg = H.PoolConfig(page_size=64, row_bytes=656, idx_dim=128, n_idx_heads=16, n_heads=heads, topk=128, n_layers=1,
                       layers_per_indexer=1, num_pages=total, num_idx_pages=1, max_requests=1, max_ctx=200064 + 128 - 200064 % 128,
                       max_q_per_req=1, hot_rows=64, max_tokens=1, idx_format=0, host_pages=1)
    host = torch.zeros(64 * 656, dtype=torch.uint8).pin_memory()
    idx = torch.zeros(8192, dtype=torch.uint8, device="cuda")
    pool = H.Pool(cfg, [kv], [idx], host)
    try:
        pool.set_pages(0, 0, block_table=table.tolist())
        work = torch.empty(pool.chunk_workspace_bytes(), dtype=torch.uint8, device="cuda")
        q = torch.randn(3, heads, 576, generator=gen, device="cuda").bfloat16()
        out = torch.empty(3, heads, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(3, heads, device="cuda")
        limit = [n, 100000, n - 1]
        pool.chunk_attention(0, i32([0, 0]), i32([0, 1, 3]), i32(limit), q, 1 / 24, out, work, lse=lse)
        assert pool.get_error() == 0
        # read back agrees with the rows too
        pos = [0, 63, 99999, 100031, 150000, n - 1]
        back = torch.empty(6, 512, device="cuda")
        pool.read_rows(0, i32([0] * 6), i32(pos), back)
    finally:
        torch.cuda.synchronize()
        pool.close()
    tab = torch.from_numpy(e4m3_to_f64(np.arange(256))).cuda()
    k = torch.cat([tab[codes.long()] * scale.double().repeat_interleave(128, 1), rope.double()], 1)
    assert torch.equal(back.double(), k[pos, :512].float().double())
    for j in range(3):
        kj = k[:limit[j]]
        z = q[j].double() @ kj.T / 24
        s = ((q[j].double().abs() @ kj.abs().T).amax(1) / 24).cpu().numpy()
        p = torch.softmax(z, 1)
        wo, a = (p @ kj[:, :512]).cpu().numpy(), (p @ kj[:, :512].abs()).cpu().numpy()
        wl = torch.logsumexp(z, 1).cpu().numpy()
        assert np.all(np.abs(out[j].double().cpu().numpy() - wo) <= CP.out_bound(wo, a, s, 2.0 ** -8, limit[j]))
        assert np.all(np.abs(lse[j].double().cpu().numpy() - wl) <= CP.lse_bound(wl, s))


def test_refusals_launch_nothing():
    rng = np.random.default_rng(30)
    with Cache(heads=16, n_layers=2, lpi=1, pages=(2,)) as c:
        H, lib = c.H, c.H.lib
        n = 4
        lat, _ = values(rng, n, 512, "bf16")
        rope, _ = values(rng, n, 64, "bf16")
        keys, _ = values(rng, n, 128, "bf16")
        req, pos = i32([0] * n), i32(range(n))
        snap = [k.clone() for k in c.kv + c.idx]

        def cache_call(fn, **kw):
            a = dict(pool=c.pool.handle, layer=0, n=n, req=req.data_ptr(), pos=pos.data_ptr(), dtype=H.BF16,
                     lat=lat.data_ptr(), ldl=512, rope=rope.data_ptr(), ldr=64, keys=keys.data_ptr(), ldk=128, ks=1.0)
            a.update(kw)
            return fn(*a.values(), torch.cuda.current_stream().cuda_stream)
        bad = [dict(pool=None), dict(layer=-1), dict(layer=2), dict(n=-1), dict(n=H.CACHE_MAX_TOKENS + 1), dict(req=None), dict(pos=None), dict(dtype=3),
               dict(dtype=-1), dict(lat=lat.data_ptr() + 2), dict(rope=rope.data_ptr() + 8), dict(keys=keys.data_ptr() + 4),
               dict(ldl=511), dict(ldl=513), dict(ldr=63), dict(ldk=127), dict(ldk=1 << 40),
               dict(lat=None, rope=None, keys=None)]
        for fn in (lib.hs_append_quantized, lib.hs_read_rows):
            for kw in bad:
                assert cache_call(fn, **kw) == INVALID, (fn, kw)
            assert cache_call(fn, n=0, req=None, pos=None, lat=None, rope=None, keys=None) == 0
        assert cache_call(lib.hs_append_quantized, lat=None) == INVALID
        assert cache_call(lib.hs_append_quantized, rope=None) == INVALID

        q = make_q(rng, n, 16, "bf16")
        out = torch.full((n, 16, 512), 0.25, dtype=torch.bfloat16, device="cuda")
        sr, ss, lim = i32([0]), i32([0, n]), i32([1] * n)

        def chunk_call(**kw):
            a = dict(pool=c.pool.handle, layer=0, n_seg=1, sr=sr.data_ptr(), ss=ss.data_ptr(), n=n, lim=lim.data_ptr(),
                     dtype=H.BF16, q=q.data_ptr(), qt=16 * 576, qh=576, sm=1.0, out=out.data_ptr(), ot=16 * 512, oh=512,
                     lse=None, work=c.work.data_ptr(), wb=c.work.numel())
            a.update(kw)
            return lib.hs_chunk_attention(*a.values(), torch.cuda.current_stream().cuda_stream)
        for kw in [dict(pool=None), dict(layer=2), dict(layer=-1), dict(n_seg=-1), dict(n_seg=H.CHUNK_MAX_SEGMENTS + 1),
                   dict(n=-1), dict(n=H.CHUNK_MAX_TOKENS + 1), dict(dtype=H.FP32), dict(sr=None), dict(ss=None),
                   dict(lim=None), dict(q=None), dict(q=q.data_ptr() + 2), dict(out=None), dict(out=out.data_ptr() + 8),
                   dict(work=None), dict(work=c.work.data_ptr() + 4), dict(wb=c.pool.chunk_workspace_bytes() - 1),
                   dict(qt=-8), dict(qt=4), dict(qh=577), dict(ot=511), dict(ot=0), dict(oh=516), dict(oh=0),
                   dict(sm=float("nan")), dict(sm=float("inf")), dict(sm=-1.01e20)]:
            assert chunk_call(**kw) == INVALID, kw
        assert chunk_call(n=0) == 0 and chunk_call(n_seg=0) == 0
        b = ctypes.c_int64(0)
        assert lib.hs_chunk_workspace(None, ctypes.byref(b)) == INVALID
        assert lib.hs_chunk_workspace(c.pool.handle, None) == INVALID
        for key_scale in (0.0, -1.0, float("nan"), float("inf"), 1e-40):     # the int8 step
            with Cache(heads=16, n_layers=1, lpi=1, pages=(1,), fmt=H.IDX_INT8) as d:
                assert cache_call(lib.hs_append_quantized, pool=d.pool.handle, ks=key_scale) == INVALID
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert c.pool.get_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(snap, c.kv + c.idx)) and torch.all(out == 0.25)


def test_prefill_then_decode_captured_replayed_and_on_another_stream():
    """The operators as they are used: a prompt in two chunks (append, attend) and a decoded
    token, captured in one graph per chunk, replayed with other inputs on a side stream; the
    decode attends through hs_sparse_mla_decode too, over the same rows."""
    rng = np.random.default_rng(40)
    with Cache(heads=64, n_layers=2, lpi=2, pages=(4,)) as c:
        s = torch.cuda.Stream()
        chunks = [(0, 100), (100, 127), (127, 128)]
        bufs, graphs = [], []
        for lo, hi in chunks:
            m = hi - lo
            proj = torch.zeros(m, 576, dtype=torch.bfloat16, device="cuda")
            b = dict(proj=proj, keys=torch.zeros(m, 128, dtype=torch.bfloat16, device="cuda"), req=i32([0] * m),
                     pos=i32(range(lo, hi)), lim=i32(range(lo + 1, hi + 1)), sr=i32([0]), ss=i32([0, m]),
                     q=torch.zeros(m, 64, 576, dtype=torch.bfloat16, device="cuda"),
                     out=torch.zeros(m, 64, 512, dtype=torch.bfloat16, device="cuda"), lse=torch.zeros(m, 64, device="cuda"))
            bufs.append(b)

        def step(b):
            c.pool.append_quantized(1, b["req"], b["pos"], b["proj"][:, :512], b["proj"][:, 512:], b["keys"])
            c.pool.chunk_attention(1, b["sr"], b["ss"], b["lim"], b["q"], 1 / 24, b["out"], c.work, lse=b["lse"])
        with torch.cuda.stream(s):
            for b in bufs:
                step(b)                                 # warm-up
        s.synchronize()
        for b in bufs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step(b)
            graphs.append(g)
        for trial in range(2):
            rows = []
            for b in bufs:
                m = b["proj"].shape[0]
                x, xf = values(rng, m, 576, "bf16", 0.3)
                b["proj"].copy_(x)
                b["keys"].copy_(values(rng, m, 128, "bf16")[0])
                b["q"].copy_(make_q(rng, m, 64, "bf16"))
                rows.append(CP.pack_rows(xf[:, :512], xf[:, 512:]))
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                for g in graphs:
                    g.replay()
            s.synchronize()
            assert c.pool.get_error() == 0
            kv = [CP.row_values(np.concatenate(rows))]
            for (lo, hi), b in zip(chunks, bufs):
                check_chunk(c, kv, [0], [0, hi - lo], np.arange(lo + 1, hi + 1), b["q"], 1 / 24, b["out"], b["lse"], "bf16")
            last = bufs[-1]
            ids = i32(c.rows_at(0, np.arange(128)))[None]
            o2, l2 = torch.zeros_like(last["out"]), torch.zeros_like(last["lse"])
            c.pool.sparse_mla_decode(1, last["q"], ids, 1 / 24, o2, l2)
            torch.cuda.synchronize()
            # two kernels of one formula: two roundings of the output to bf16 (2^-8 of the value
            # each), P rounded to bf16 there (2^-8 of sum p |v|), and this call's own bound
            qf = last["q"][0].float().cpu().numpy().astype(np.float64)
            wo, wl, a, sz = CP.attend(qf, kv[0], 1 / 24)
            bound = 2 * CP.out_bound(wo, a, sz, HALF_STEP["bf16"], 128) + 2.0 ** -8 * a
            assert np.all((o2[0].float() - last["out"][0].float()).abs().cpu().numpy() <= bound)
            assert np.all((l2[0] - last["lse"][0]).abs().cpu().numpy() <= 2 * CP.lse_bound(wl, sz))
