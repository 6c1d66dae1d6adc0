"""Argument checks of the cache operators that need no GPU: the C entry points without a pool,
and the binding's checks of shapes, types, strides and devices."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def H():
    from sparse_mla_kv_indexer_gb300 import build
    build.build()
    from sparse_mla_kv_indexer_gb300 import hisparse
    return hisparse


class FakePool:
    """A Pool without a library handle, on 'device' -1 (the CPU): every check runs, no call
    gets past the library's own (a NULL pool is HS_ERR_INVALID)."""

    def __new__(cls, H, heads=16):
        p = H.Pool.__new__(H.Pool)
        p.cfg = H.PoolConfig(n_heads=heads)
        p.handle = None
        p.device = -1
        return p


def test_null_pool_is_refused(H):
    P = ctypes.c_void_p
    assert H.lib.hs_append_quantized(None, 0, 1, P(16), P(16), 0, P(16), 512, P(16), 64, None, 0, 1.0, None) == 1
    assert H.lib.hs_read_rows(None, 0, 1, P(16), P(16), 0, P(16), 512, P(16), 64, None, 0, 1.0, None) == 1
    assert H.lib.hs_chunk_attention(None, 0, 1, P(16), P(16), 1, P(16), 0, P(16), 9216, 576, 1.0, P(16), 8192, 512,
                                    None, P(16), 1 << 30, None) == 1
    n = ctypes.c_int64(0)
    assert H.lib.hs_chunk_workspace(None, ctypes.byref(n)) == 1


def test_constants_match_the_header(H):
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "hisparse.h")).read()
    for name, want in [("HS_BF16", H.BF16), ("HS_FP16", H.FP16), ("HS_FP32", H.FP32),
                       ("HS_CACHE_MAX_TOKENS", H.CACHE_MAX_TOKENS),
                       ("HS_CHUNK_MAX_SEGMENTS", H.CHUNK_MAX_SEGMENTS), ("HS_CHUNK_MAX_TOKENS", H.CHUNK_MAX_TOKENS)]:
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == want


def test_the_binding_checks_cache_arguments(H):
    p = FakePool(H)
    i = torch.zeros(3, dtype=torch.int32)
    lat, rope, keys = torch.zeros(3, 512), torch.zeros(3, 64), torch.zeros(3, 128)
    for call in (p.append_quantized, p.read_rows):
        for args in [(i, i), (i.long(), i, lat, rope), (i, i[:2], lat, rope), (i.float(), i, lat, rope),
                     (i, i, lat[:2], rope), (i, i, lat, lat), (i, i, lat, rope.half()), (i, i, lat.double(), rope.double()),
                     (i, i, lat, rope, rope), (i, i, torch.zeros(512, 3).t(), rope), (i, i, lat[None], rope)]:
            with pytest.raises(ValueError):
                call(0, *args, stream=0)
        with pytest.raises(H.HisparseError):     # well-formed: the library refuses the NULL pool
            call(0, i, i, lat, rope, keys, stream=0)
        p.device = 0
        with pytest.raises(ValueError):          # a CPU tensor on a pool of cuda:0
            call(0, i, i, lat, rope, keys, stream=0)
        p.device = -1


def test_the_binding_checks_attention_arguments(H):
    p = FakePool(H)
    ok = dict(seg_req=torch.zeros(1, dtype=torch.int32), seg_start=torch.zeros(2, dtype=torch.int32),
              limit=torch.ones(3, dtype=torch.int32), q=torch.zeros(3, 16, 576, dtype=torch.bfloat16), sm_scale=1.0,
              out=torch.zeros(3, 16, 512, dtype=torch.bfloat16), work=torch.zeros(64, dtype=torch.uint8),
              lse=torch.zeros(3, 16))
    with pytest.raises(H.HisparseError):
        p.chunk_attention(0, **ok, stream=0)
    for bad in [dict(q=torch.zeros(3, 16, 576)), dict(q=torch.zeros(3, 32, 576, dtype=torch.bfloat16)),
                dict(q=torch.zeros(2, 16, 576, dtype=torch.bfloat16)), dict(out=torch.zeros(3, 16, 512, dtype=torch.float16)),
                dict(out=torch.zeros(3, 16, 576, dtype=torch.bfloat16)), dict(lse=torch.zeros(3, 15)),
                dict(lse=torch.zeros(3, 16, dtype=torch.float16)), dict(lse=torch.zeros(16, 3).t()),
                dict(seg_start=torch.zeros(1, dtype=torch.int32)), dict(seg_req=torch.zeros(1, dtype=torch.int64)),
                dict(limit=torch.ones(3)), dict(work=torch.zeros(64, 2, dtype=torch.uint8)[:, 0]),
                dict(q=torch.zeros(3, 576, 16, dtype=torch.bfloat16).transpose(1, 2))]:
        with pytest.raises(ValueError):
            p.chunk_attention(0, **{**ok, **bad}, stream=0)
    p.device = 0
    with pytest.raises(ValueError):
        p.chunk_attention(0, **ok, stream=0)
