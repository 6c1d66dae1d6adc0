"""Argument checks of the operators around a shared cache that need no GPU: the C entry points without
a pool, and the binding's checks of shapes, types, strides and devices."""
import ctypes
import os
import re

import pytest

from test_cache_ops_args import FakePool, H, torch  # noqa: F401  (H is the fixture)

P = ctypes.c_void_p


def test_null_pool_is_refused(H):
    lib, part = H.lib, (H.RotaryPart * 1)()
    assert lib.hs_rotary(None, 1, P(16), 64, P(16), 1.0, 0, 0, 1, part, None) == 1
    assert lib.hs_fork_requests(None, 1, P(16), P(16), P(16), P(16), P(16), None) == 1
    assert lib.hs_copy_pages(None, 1, P(16), P(16), 0, None, None, 0, None) == 1
    assert lib.hs_get_pages(None, 1, P(16), 0, 1, P(16), None, None, None) == 1
    assert lib.hs_prefix_attention(None, 0, 1, P(16), P(16), 1, P(16), P(16), 1, P(16), 0, P(16), 9216, 576, 1.0, P(16), 8192,
                                   512, None, P(16), 1 << 40, None) == 1
    n = ctypes.c_int64(0)
    assert lib.hs_prefix_workspace(None, 1, 1, 1, ctypes.byref(n)) == 1


def test_constants_match_the_header(H):
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "hisparse.h")).read()
    for name, want in [("HS_COPY_MAX_PAGES", H.COPY_MAX_PAGES), ("HS_ROTARY_MAX_DIMS", H.ROTARY_MAX_DIMS),
                       ("HS_ROTARY_MAX_HEADS", H.ROTARY_MAX_HEADS), ("HS_ROTARY_MAX_PARTS", H.ROTARY_MAX_PARTS),
                       ("HS_PREFIX_MAX_GROUPS", H.PREFIX_MAX_GROUPS), ("HS_PREFIX_MAX_TOKENS", H.PREFIX_MAX_TOKENS),
                       ("HS_ROTARY_PAIRS", H.ROTARY_LAYOUTS["pairs"]), ("HS_ROTARY_HALVES", H.ROTARY_LAYOUTS["halves"])] + \
                      [("HS_ROTARY_" + k.upper(), v) for k, v in H.ROTARY_SCALINGS.items()]:
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == want


def test_the_binding_checks_rotary_arguments(H):
    p = FakePool(H)
    x, o = torch.zeros(3, 4, 64), torch.zeros(3, 4, 64)
    ok = dict(pos=torch.zeros(3, dtype=torch.int32), steps=torch.zeros(32, dtype=torch.int64), parts=[(x, o, "pairs")])
    with pytest.raises(H.HisparseError):
        p.rotary(**ok, stream=0)
    with pytest.raises(H.HisparseError):
        p.rotary(**{**ok, "parts": [(x, x, "halves"), (x[:, 0], o[:, 0], "pairs")]}, stream=0)
    for bad in [dict(parts=[]), dict(parts=ok["parts"] * 5), dict(parts=[(x, o, "other")]), dict(parts=[(x, o[:2], "pairs")]),
                dict(parts=[(x[:2], o[:2], "pairs")]), dict(parts=[(x, o.half(), "pairs")]), dict(parts=[(x.double(), o.double(), "pairs")]),
                dict(parts=[(x, o, "pairs"), (x[:, :, :32], o[:, :, :32], "pairs")]), dict(parts=[(x[0], o[0], "pairs")]),
                dict(parts=[(torch.zeros(3, 64, 4).transpose(1, 2), o, "pairs")]), dict(parts=[(x[None], o[None], "pairs")]),
                dict(pos=torch.zeros(3, dtype=torch.int64)), dict(pos=torch.zeros(6, dtype=torch.int32)[::2]),
                dict(steps=torch.zeros(64, dtype=torch.int64)), dict(steps=torch.zeros(32, dtype=torch.int32)),
                dict(steps=torch.zeros(64, dtype=torch.int64)[::2])]:
        with pytest.raises(ValueError):
            p.rotary(**{**ok, **bad}, stream=0)
    p.device = 0
    with pytest.raises(ValueError):
        p.rotary(**ok, stream=0)


def test_the_binding_checks_page_arguments(H):
    p = FakePool(H)
    i, two = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for args in [(i, i, i, i, i), (i, i, i, i)]:
        with pytest.raises(H.HisparseError):
            p.fork_requests(*args, stream=0)
    for k in range(5):
        for bad in (two, i.long(), torch.zeros(6, dtype=torch.int32)[::2]):
            args = [i] * 5
            args[k] = bad
            if k == 0 and bad is two:
                continue
            with pytest.raises(ValueError):
                p.fork_requests(*args, stream=0)
    with pytest.raises(H.HisparseError):
        p.copy_pages(i, i, two, two, remap=True, stream=0)
    for args in [(i,), (i, None, i, i), (i, two), (i, i, two, i), (i.long(), i.long()), (i, i, None, two)]:
        with pytest.raises(ValueError):
            p.copy_pages(*args, stream=0)
    bt, host = torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, 5, dtype=torch.int64)
    with pytest.raises(H.HisparseError):
        p.get_pages(i, 0, bt, bt, host, stream=0)
    for args in [(i, 0), (i, 0, host), (i, 0, bt, None, bt), (two, 0, bt), (i, 0, bt, bt[:, :4]), (i, 0, bt[:, ::2]), (i.long(), 0, bt)]:
        with pytest.raises(ValueError):
            p.get_pages(*args, stream=0)
    p.device = 0
    for call in (lambda: p.fork_requests(i, i, i, i, i, stream=0), lambda: p.copy_pages(i, i, stream=0),
                 lambda: p.get_pages(i, 0, bt, stream=0)):
        with pytest.raises(ValueError):
            call()


def test_the_binding_checks_prefix_arguments(H):
    p = FakePool(H)
    ok = dict(group_start=torch.zeros(2, dtype=torch.int32), group_len=torch.zeros(1, dtype=torch.int32),
              seg_req=torch.zeros(1, dtype=torch.int32), seg_start=torch.zeros(2, dtype=torch.int32),
              limit=torch.ones(3, dtype=torch.int32), q=torch.zeros(3, 16, 576, dtype=torch.bfloat16), sm_scale=1.0,
              out=torch.zeros(3, 16, 512, dtype=torch.bfloat16), work=torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(H.HisparseError):
        p.prefix_attention(0, **ok, stream=0)
    for bad in [dict(group_start=torch.zeros(1, dtype=torch.int32)), dict(group_len=torch.zeros(1, dtype=torch.int64)),
                dict(group_len=torch.zeros(2, dtype=torch.int32)), dict(q=torch.zeros(3, 16, 576)),
                dict(out=torch.zeros(3, 16, 512, dtype=torch.float16)), dict(lse=torch.zeros(3, 15)),
                dict(seg_start=torch.zeros(1, dtype=torch.int32))]:
        with pytest.raises(ValueError):
            p.prefix_attention(0, **{**ok, **bad}, stream=0)
