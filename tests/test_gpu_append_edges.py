"""Edges of the quantised append on the GPU: positions given more than once."""
import numpy as np
import pytest

import cache_plain as CP
from test_gpu_cache_ops import RANGE, Cache, dt, i32, torch, values

pytestmark = pytest.mark.gpu


def chains(rng, n, pages, longest):
    """Positions that occur in up to four tokens, with up to `longest` padding tokens between one
    and the next; returns req, pos and the token that each position is written from."""
    req, pos, last = [], [], {}
    free = iter(rng.permutation(pages * 64))
    while len(req) < n:
        p = int(next(free))
        for k in range(int(rng.integers(1, 5))):
            if k:
                gap = int(rng.integers(0, longest + 1))
                req += [-1] * gap
                pos += rng.integers(0, pages * 64, gap).tolist()
            last[p] = len(req)
            req.append(0)
            pos.append(p)
    return np.array(req, np.int32), np.array(pos, np.int32), last


@pytest.mark.parametrize("n,longest", [(40, 0), (300, 2), (3000, 31), (3000, 3), (9000, 5), (40000, 31), (200000, 2)])
def test_a_position_given_again_behind_padding_is_written_from_the_later_token(n, longest):
    rng = np.random.default_rng(n + longest)
    pages = -(-n // 64)
    req, pos, last = chains(rng, n, pages, longest)
    n = len(req)
    with Cache(n_layers=1, lpi=1, pages=(pages,)) as c:
        lat, lf = values(rng, n, 512, "bf16")
        rope, rf = values(rng, n, 64, "bf16")
        keys, kf = values(rng, n, 128, "bf16")
        c.pool.append_quantized(0, i32(req), i32(pos), lat, rope, keys)
        assert c.pool.get_error() == 0
        at, tok = np.array(list(last)), np.array(list(last.values()))
        some = np.sort(rng.permutation(len(at))[:20000])
        at, tok = at[some], tok[some]
        assert np.array_equal(c.get_rows(0, 0, at), CP.pack_rows(lf[tok], rf[tok]))
        codes, scales = c.get_keys(0, 0, at)
        wc, ws = CP.quantise(kf[tok])
        assert np.array_equal(codes, wc) and np.array_equal(scales, ws[:, 0])


def test_the_last_of_32_padding_tokens_apart():
    """31 padding tokens between: one write; a chain over a warp's and a call's end."""
    rng = np.random.default_rng(1)
    with Cache(n_layers=1, lpi=1, pages=(4,)) as c:
        for lead in (0, 1, 30, 31, 32, 33):
            n = lead + 33
            req, pos = np.full(n, -1, np.int32), np.arange(n, dtype=np.int32)
            req[:lead + 1] = 0
            req[-1], pos[-1] = 0, lead
            lat, lf = values(rng, n, 512, "bf16")
            rope, rf = values(rng, n, 64, "bf16")
            c.pool.append_quantized(0, i32(req), i32(pos), lat, rope)
            assert c.pool.get_error() == 0
            tok = np.r_[np.arange(lead), n - 1]
            assert np.array_equal(c.get_rows(0, 0, np.arange(lead + 1)), CP.pack_rows(lf[tok], rf[tok]))


@pytest.mark.parametrize("magnitude", [0.0, 1e-45, 1e-40, 1e-37, 5e-36, 1e-20, 1.0, 3.3e38])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_an_infinity_is_the_largest_code_whatever_the_group(dtype, magnitude):
    """In groups whose scale is held at 2^-126 too; the finite values beside it keep the group's
    scale, which is 1 where they are all zero."""
    rng = np.random.default_rng(5)
    with Cache(pages=(2,)) as c:
        x = rng.uniform(-1, 1, (3, 512)) * magnitude
        x[:, ::128] = magnitude
        x[1, 7], x[1, 200], x[2, 300], x[2, 301] = np.inf, -np.inf, np.inf, np.nan
        k = rng.uniform(-1, 1, (3, 128)) * magnitude
        k[2, 100] = -np.inf
        lat, keys = (torch.from_numpy(v.astype(np.float32)).to(dt(dtype)).cuda() for v in (x, k))
        rope = torch.zeros(3, 64, dtype=dt(dtype), device="cuda")
        c.pool.append_quantized(0, i32([0, 0, 0]), i32([0, 1, 64]), lat, rope, keys)
        assert c.pool.get_error() == RANGE
        lf, kf = lat.float().cpu().numpy(), keys.float().cpu().numpy()
        want = CP.pack_rows(np.where(np.isfinite(lf), lf, 0), np.zeros((3, 64)))
        want[1, 7], want[1, 200], want[2, 300], want[2, 301] = 0x7E, 0xFE, 0x7E, 0
        assert np.array_equal(c.get_rows(0, 0, [0, 1, 64]), want)
        codes, scales = c.get_keys(0, 0, [0, 1, 64])
        wc, ws = CP.quantise(np.where(np.isfinite(kf), kf, 0))
        wc[2, 100] = 0xFE
        assert np.array_equal(codes, wc) and np.array_equal(scales, ws[:, 0])


def test_finite_rope_beyond_bf16_is_the_largest_value_and_reported():
    """fp32 rope from bf16's largest value and half a step on; the value below it is rounded."""
    with Cache(pages=(2,)) as c:
        top = np.array([0x7F7F0000, 0x7F7F7FFF, 0x7F7F8000, 0x7F7FFFFF], np.uint32).view(np.float32)
        lat = torch.ones(1, 512, device="cuda")
        for i, v in enumerate(top):
            for sign in (1.0, -1.0):
                rope = torch.zeros(1, 64, device="cuda")
                rope[0, 9] = float(v) * sign
                c.pool.append_quantized(0, i32([0]), i32([5]), lat, rope)
                assert c.pool.get_error() == (RANGE if i >= 2 else 0), hex(v.view(np.uint32))
                got = c.get_rows(0, 0, [5])[0, 528:].view("<u2")
                assert got[9] == (0x7F7F if sign > 0 else 0xFF7F) and np.all(np.delete(got, 9) == 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_minus_zero_keeps_its_sign(dtype):
    """The e4m3 value nearest to -0 / scale is -0, in groups of zeros and beside other values."""
    rng = np.random.default_rng(6)
    with Cache(pages=(1,)) as c:
        x = rng.standard_normal((2, 640)).astype(np.float32)
        x[:, 128:256] = 0
        x[1, 512:] = 0
        x[rng.random((2, 640)) < 0.3] = 0
        x = np.where((x == 0) & (rng.random((2, 640)) < 0.5), np.float32(-0.0), x)
        t = torch.from_numpy(x).to(dt(dtype)).cuda()
        rope = torch.zeros(2, 64, dtype=dt(dtype), device="cuda")
        c.pool.append_quantized(0, i32([0, 0]), i32([3, 4]), t[:, :512], rope, t[:, 512:])
        assert c.pool.get_error() == 0
        f = t.float().cpu().numpy()
        assert np.array_equal(c.get_rows(0, 0, [3, 4]), CP.pack_rows(f[:, :512], np.zeros((2, 64))))
        codes, scales = c.get_keys(0, 0, [3, 4])
        wc, ws = CP.quantise(f[:, 512:])
        assert np.array_equal(codes, wc) and np.array_equal(scales, ws[:, 0])
