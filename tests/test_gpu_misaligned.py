"""Addresses of 4-byte words that are not multiples of 4: refused on the host by the cache
operators' C entry points."""
import pytest

from test_gpu_cache_ops import INVALID, Cache, i32, torch

pytestmark = pytest.mark.gpu


def test_misaligned_words_are_refused():
    with Cache(heads=16, n_layers=1, lpi=1, pages=(2,)) as c:
        lib, H, st = c.H.lib, c.H, torch.cuda.current_stream().cuda_stream
        ids = i32([0] * 16)
        lat = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
        rope = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
        at = ids.data_ptr()
        before = [k.clone() for k in c.kv]
        for fn in (lib.hs_append_quantized, lib.hs_read_rows):
            for req, pos in ((at + 2, at), (at, at + 1), (at + 3, at + 3)):
                assert fn(c.pool.handle, 0, 2, req, pos, H.BF16, lat.data_ptr(), 512, rope.data_ptr(), 64, None, 0, 1.0,
                          st) == INVALID
        q = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device="cuda")
        out = torch.full((2, 16, 512), 0.25, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((40,), 0.25, device="cuda")
        for k in range(4):
            words = [at, at, at, lse.data_ptr()]
            words[k] += 2
            assert lib.hs_chunk_attention(c.pool.handle, 0, 1, words[0], words[1], 2, words[2], H.BF16, q.data_ptr(), 9216, 576,
                                          1.0, out.data_ptr(), 8192, 512, words[3], c.work.data_ptr(), c.work.numel(),
                                          st) == INVALID, k
        torch.cuda.synchronize()
        assert c.pool.get_error() == 0 and torch.all(out == 0.25) and torch.all(lse == 0.25)
        assert all(torch.equal(a, b) for a, b in zip(before, c.kv))
