"""Rotary positions on the GPU against plain 64-bit arithmetic: layouts, types, strides, sizes, far
positions, and the calls that are refused."""
import math

import numpy as np
import pytest

from test_gpu_cache_ops import INVALID, Cache, dt, i32, torch

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}   # half a step of the smallest values


@pytest.fixture(scope="module")
def pool():
    with Cache(heads=16, n_layers=1, lpi=1, pages=(2,)) as c:
        yield c.pool


def angles(pos, steps):
    """Exact phases of positions, in radians as doubles (off by 2^-53 of a turn)."""
    out = np.empty((len(pos), len(steps)))
    for j, p in enumerate(np.asarray(pos).tolist()):
        for i, s in enumerate(steps.tolist()):
            out[j, i] = (p * s) % (1 << 64) / 2.0 ** 64 * 2 * math.pi
    return out


def rotated(x, w, layout, magnitude=1.0, inverse=False):
    """x [n, heads, dims] in 64 bits, and |a| + |b| of every pair at both of its places."""
    if inverse:
        w = -w
    c, s = np.cos(w)[:, None] * magnitude, np.sin(w)[:, None] * magnitude
    half = x.shape[2] // 2
    a, b = (x[:, :, 0::2], x[:, :, 1::2]) if layout == "pairs" else (x[:, :, :half], x[:, :, half:])
    out, size = np.empty_like(x), np.empty_like(x)
    ra, rb, sz = a * c - b * s, a * s + b * c, np.abs(a) + np.abs(b)
    if layout == "pairs":
        out[:, :, 0::2], out[:, :, 1::2], size[:, :, 0::2], size[:, :, 1::2] = ra, rb, sz, sz
    else:
        out[:, :, :half], out[:, :, half:], size[:, :, :half], size[:, :, half:] = ra, rb, sz, sz
    return out, size


def bound(want, size, dtype, magnitude=1.0):
    """A cosine or sine: the phase cut to 2^-32 turns (2^-29.3), the remaining eighth of a turn rounded to 24
    bits (2^-24.3), sincospi within 2 units of 2^-24: below 1.5 * 2^-23 in all; times the magnitude, the
    products and their sum rounded to fp32 each (2^-24 of magnitude * size): below 3 * 2^-23; then one rounding
    to the type."""
    return 3 * 2.0 ** -23 * magnitude * size + 1.001 * HALF_STEP[dtype] * np.abs(want) + LEAST[dtype]


def check(got, x, w, layout, dtype, magnitude=1.0, inverse=False):
    x3 = x.double().cpu().numpy()
    x3 = x3[:, None] if x3.ndim == 2 else x3
    want, size = rotated(x3, w, layout, magnitude, inverse)
    g = got.double().cpu().numpy()
    g = g[:, None] if g.ndim == 2 else g
    err, b = np.abs(g - want), bound(want, size, dtype, magnitude)
    assert np.all(err <= b), (float((err / b).max()), float(err.max()))


def randn(rng, *shape, dtype="fp32"):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt(dtype)).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("dims", [2, 6, 16, 20, 64, 96, 256])
@pytest.mark.parametrize("n,heads", [(1, 1), (1, 64), (5, 3), (333, 2), (40, 16)])
def test_every_layout_type_and_size(pool, dtype, layout, dims, n, heads):
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    rng = np.random.default_rng(dims + n)
    steps, m = H.rotary_steps(dims, 10000.0, "ramp" if dims > 2 else "none", factor=40.0, original_ctx=4096.0, magnitude=0.1)
    pos = rng.integers(0, 1 << 20, n)
    x, out = randn(rng, n, heads, dims, dtype=dtype), torch.full((n, heads, dims), 7.0, dtype=dt(dtype), device="cuda")
    pool.rotary(i32(pos), steps.cuda(), [(x, out, layout)], magnitude=m)
    w = angles(pos, steps)
    check(out, x, w, layout, dtype, m)
    # in place, turned back: the transpose
    again = out.clone()
    pool.rotary(i32(pos), steps.cuda(), [(out, out, layout)], magnitude=1.0, inverse=True)
    check(out, again, w, layout, dtype, 1.0, True)
    assert pool.get_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_four_parts_of_strided_tensors(pool, dtype, shift):
    """Parts of heads, at addresses that 16-byte accesses reach and at others; what lies around stays."""
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    rng = np.random.default_rng(shift)
    n, d = 37, 64
    steps, _ = H.rotary_steps(d, 10000.0)
    pos = np.arange(n) + 100000
    up, q = randn(rng, n, 16, 200, dtype=dtype), torch.full((n, 16, 640), 7.0, dtype=dt(dtype), device="cuda")
    down, rope = randn(rng, n, 640, dtype=dtype), torch.full((n, 72), 7.0, dtype=dt(dtype), device="cuda")
    iq, ik = randn(rng, n, 5, 136, dtype=dtype), randn(rng, n, 136, dtype=dtype)
    iq0, ik0 = iq.clone(), ik.clone()
    at = lambda t: t[..., shift:shift + d]  # noqa: E731
    pool.rotary(i32(pos), steps.cuda(), [(at(up[:, :, 120:]), at(q[:, :, 512:]), "pairs"), (at(down[:, 512:]), at(rope), "halves"),
                                         (at(iq), at(iq), "halves"), (at(ik), at(ik), "pairs")])
    w = angles(pos, steps)
    check(at(q[:, :, 512:]), at(up[:, :, 120:]), w, "pairs", dtype)
    check(at(rope), at(down[:, 512:]), w, "halves", dtype)
    check(at(iq), at(iq0), w, "halves", dtype)
    check(at(ik), at(ik0), w, "pairs", dtype)
    for t, t0, lo in ((q, None, 512), (rope, None, 0), (iq, iq0, 0), (ik, ik0, 0)):
        keep = torch.ones(t.shape[-1], dtype=torch.bool)
        keep[lo + shift:lo + shift + d] = False
        assert torch.equal(t[..., keep], torch.full_like(t, 7.0)[..., keep] if t0 is None else t0[..., keep])


def test_positions_at_the_ends_of_their_range(pool):
    """Every quarter and eighth of a turn from whole-number steps, and the largest, the least and negative
    positions, whose angles are exact however far they are."""
    rng = np.random.default_rng(5)
    steps = torch.tensor([1 << 61, 1 << 62, (1 << 61) - 1, (1 << 61) + (1 << 32), 1 << 31, 0x123456789ABCDEF, 3, 0], dtype=torch.int64)
    pos = np.array([0, 1, 2, 3, 4, 5, 6, 7, 8, -1, -2, -7, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 1310719])
    x, out = randn(rng, len(pos), 3, 16), torch.zeros(len(pos), 3, 16, device="cuda")
    pool.rotary(i32(pos), steps.cuda(), [(x, out, "halves")])
    check(out, x, angles(pos, steps), "halves", "fp32")
    assert torch.equal(out[0], x[0])                      # position 0 turns by nothing, exactly
    assert torch.equal(out[:, :, 7], x[:, :, 7]) and torch.equal(out[:, :, 15], x[:, :, 15])


def test_values_that_are_not_finite_stay_in_their_pair(pool):
    rng = np.random.default_rng(6)
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    steps, _ = H.rotary_steps(64, 10000.0)
    x = randn(rng, 4, 2, 64, dtype="fp16")
    x[1, 0, 10], x[2, 1, 40], x[3, 0, 0] = float("nan"), float("inf"), 65504.0
    x[3, 0, 32] = 65504.0
    out = torch.zeros_like(x)
    pool.rotary(i32([1, 2, 3, 4]), steps.cuda(), [(x, out, "halves")])
    nan = ~torch.isfinite(out)
    assert nan[1, 0, 10] and nan[1, 0, 42] and nan[2, 1, 8] and nan[2, 1, 40]
    assert torch.isinf(out[3, 0, 0]) or torch.isinf(out[3, 0, 32])   # |cos| + |sin| > 1 at 4 radians
    nan[1, 0, [10, 42]] = nan[2, 1, [8, 40]] = nan[3, 0, [0, 32]] = False
    assert not nan.any() and pool.get_error() == 0


def test_a_broadcast_input_and_no_tokens(pool):
    rng = np.random.default_rng(7)
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    steps, _ = H.rotary_steps(32, 500.0)
    one = randn(rng, 9, 1, 32, dtype="bf16")
    out = torch.zeros(9, 6, 32, dtype=torch.bfloat16, device="cuda")
    pool.rotary(i32(range(9)), steps.cuda(), [(one.expand(9, 6, 32), out, "pairs")])
    check(out, one.expand(9, 6, 32), angles(range(9), steps), "pairs", "bf16")
    pool.rotary(i32([]), steps.cuda(), [(one[:0], out[:0, :1], "pairs")])


def test_large_calls_and_offsets_beyond_32_bits(pool):
    """The most tokens of a call, two dims each, whose last values lie behind 2^32 bytes; and many tokens of
    many heads against a plain form on the GPU."""
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    n = H.CACHE_MAX_TOKENS
    wide = torch.zeros(n, 144, dtype=torch.bfloat16, device="cuda")
    x = wide[:, 140:142]
    x[:, 0] = 1.0
    pos = torch.arange(n, dtype=torch.int32, device="cuda") % 8
    steps = torch.tensor([1 << 61], dtype=torch.int64, device="cuda")      # an eighth of a turn
    pool.rotary(pos, steps, [(x, x, "pairs")])
    r = 2.0 ** 0.5 / 2
    want = torch.tensor([[1, 0], [r, r], [0, 1], [-r, r], [-1, 0], [-r, -r], [0, -1], [r, -r]], device="cuda").bfloat16()
    for a in range(0, n, 1 << 21):
        assert torch.equal(x[a:a + (1 << 21)], want.repeat((1 << 18), 1)), a
    assert not wide[:, :140].any() and not wide[:, 142:].any()
    with pytest.raises(H.HisparseError):
        more = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        y = torch.zeros(n + 1, 2, device="cuda")
        pool.rotary(more, steps, [(y, y, "pairs")])
    del wide, x
    g = torch.Generator("cuda").manual_seed(1)
    n = 5003
    q = torch.randn(n, 64, 64, generator=g, device="cuda")
    steps, _ = H.rotary_steps(64, 10000.0)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    pool.rotary(pos, steps.cuda(), [(q, out, "pairs")])
    w = pos.double()[:, None, None] * (10000.0 ** (-torch.arange(32, device="cuda").double() / 32))
    a, b = q[..., 0::2].double(), q[..., 1::2].double()
    want = torch.stack([a * w.cos() - b * w.sin(), a * w.sin() + b * w.cos()], -1).flatten(-2)
    # 2^20 radians in 64 bits are off by 2^-33
    limit = 3.1 * 2.0 ** -23 * (a.abs() + b.abs()).repeat_interleave(2, -1) + 1.001 * 2.0 ** -24 * want.abs()
    assert torch.all((out.double() - want).abs() <= limit)


def test_refusals(pool):
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    lib, st = H.lib, torch.cuda.current_stream().cuda_stream
    x = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(x, 7.0)
    pos, steps = i32([0] * 4), torch.zeros(32, dtype=torch.int64, device="cuda")

    def call(n=4, pos_at=pos.data_ptr(), dims=64, steps_at=steps.data_ptr(), magnitude=1.0, dtype=0, n_parts=1, **part):
        p = (H.RotaryPart * 4)()
        for k in range(4):
            f = dict(d_in=x.data_ptr(), d_out=o.data_ptr(), in_stride_token=256, in_stride_head=64, out_stride_token=256,
                     out_stride_head=64, heads=4, layout=0)
            f.update(part)
            for name, v in f.items():
                setattr(p[k], name, v)
        return lib.hs_rotary(pool.handle, n, pos_at, dims, steps_at, magnitude, 0, dtype, n_parts, p, st)

    for bad in [dict(n=-1), dict(n=(1 << 24) + 1), dict(pos_at=None), dict(pos_at=pos.data_ptr() + 2), dict(dims=0), dict(dims=63),
                dict(dims=258), dict(steps_at=None), dict(steps_at=steps.data_ptr() + 4), dict(magnitude=float("nan")),
                dict(magnitude=float("inf")), dict(dtype=3), dict(dtype=-1), dict(n_parts=0), dict(n_parts=5), dict(heads=0),
                dict(heads=1025), dict(layout=2), dict(layout=-1), dict(d_in=None), dict(d_out=None), dict(d_in=x.data_ptr() + 1),
                dict(d_out=o.data_ptr() + 1), dict(in_stride_token=-1), dict(in_stride_head=-64), dict(out_stride_token=63),
                dict(out_stride_head=63), dict(out_stride_token=1 << 40), dict(d_in=o.data_ptr(), in_stride_token=512),
                dict(d_in=o.data_ptr(), in_stride_head=128)]:
        assert call(**bad) == INVALID, bad
    assert lib.hs_rotary(pool.handle, 4, pos.data_ptr(), 64, steps.data_ptr(), 1.0, 0, 0, 1, None, st) == INVALID
    torch.cuda.synchronize()
    assert torch.all(o == 7.0) and pool.get_error() == 0
    assert call() == 0 and call(n=0, pos_at=None) == 0
    torch.cuda.synchronize()
    assert not o.any()
