"""Reading back positions of which a part is missing, on the GPU."""
import numpy as np
import pytest

import cache_plain as CP
from test_gpu_cache_ops import BAD_ID, HOST_MISSING, Cache, i32, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_token_with_a_missing_part_is_left_alone_whole(fmt):
    """A row that is nowhere, an index-key page that is nowhere, both: none of the token's outputs
    is written, whichever are asked for, the others' are, and the row's error comes first."""
    rng = np.random.default_rng(1)
    with Cache(pages=(4,), fmt=fmt) as c:
        rows = CP.pack_rows(rng.standard_normal((256, 512)), rng.standard_normal((256, 64)))
        c.put_rows(0, 0, np.arange(256), rows)
        c.idx[0].copy_(torch.from_numpy(rng.integers(0, 40, (c.n_pages, c.page_bytes), dtype=np.uint8)))
        pos = i32([3, 70, 130, 200])

        def read(order=(0, 1, 2, 3), **parts):
            got = {k: torch.full((len(order), w), 7.0, device="cuda")
                   for k, w in (("latent", 512), ("rope", 64), ("keys", 128)) if parts.get(k, True)}
            c.pool.read_rows(0, i32([0] * len(order)), pos[list(order)].contiguous(), **got, key_scale=0.5)
            return c.pool.get_error(), got
        err, whole = read()
        assert err == 0
        c.pool.set_pages(0, 1, block_table=[-1])       # position 70: no row, no host copy
        c.pool.set_pages(0, 2, idx_pages=[-1])         # position 130: no key page
        c.pool.set_pages(0, 3, block_table=[-1], idx_pages=[-1])
        err, got = read()
        assert err in (HOST_MISSING, BAD_ID)
        for k in whole:
            assert torch.equal(got[k][0], whole[k][0]) and torch.all(got[k][1:] == 7.0), k
        for order, want in [((0, 1), HOST_MISSING), ((2, 0), BAD_ID), ((0, 3), HOST_MISSING)]:
            assert read(order)[0] == want, order
        err, got = read(latent=False, rope=False)      # the keys alone
        assert err == BAD_ID
        assert torch.equal(got["keys"][:2], whole["keys"][:2]) and torch.all(got["keys"][2:] == 7.0)
        err, got = read(keys=False)                    # the rows alone
        assert err == HOST_MISSING
        for k in ("latent", "rope"):
            assert torch.equal(got[k][[0, 2]], whole[k][[0, 2]]) and torch.all(got[k][[1, 3]] == 7.0)
