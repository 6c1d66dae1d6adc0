"""A Pool takes raw addresses, and is made and used without torch; the calls on tensors find the
pool's device when they are first made."""
import sys

import numpy as np
import pytest


@pytest.fixture(scope="module")
def H():
    from sparse_mla_kv_indexer_gb300 import build
    build.build()
    from sparse_mla_kv_indexer_gb300 import hisparse
    return hisparse


def test_the_constructor_reaches_the_library(H, monkeypatch):
    """Addresses that the library's own check of the geometry refuses before it reads them."""
    monkeypatch.setitem(sys.modules, "torch", None)    # import torch fails
    with pytest.raises(H.HisparseError):
        H.Pool(H.PoolConfig(), [16], [16], 16)


def test_the_device_is_looked_up_once(H, monkeypatch):
    p = H.Pool.__new__(H.Pool)
    p.cfg, p.handle, p.device = H.PoolConfig(n_heads=16), None, None
    with pytest.raises(H.HisparseError):               # the library's refusal: no pool, or another device's
        p._device()
    assert p.device is None                            # nothing was settled
    asked = []
    monkeypatch.setattr(p, "chunk_workspace_bytes", lambda: asked.append(1) or 0, raising=False)
    monkeypatch.setattr(H, "_current_device", lambda: 3)
    assert p._device() == 3 and p._device() == 3 and asked == [1]


@pytest.mark.gpu
def test_a_pool_of_raw_addresses_made_without_torch(H, monkeypatch):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import cache_plain as CP
    kv = torch.zeros(4 * 64, 656, dtype=torch.uint8, device="cuda")
    idx = torch.zeros(4, 8448, dtype=torch.uint8, device="cuda")
    host = torch.zeros(64 * 656, dtype=torch.uint8).pin_memory()
    torch.cuda.synchronize()
    cfg = H.PoolConfig(page_size=64, row_bytes=656, idx_dim=128, n_idx_heads=16, n_heads=16, topk=128, n_layers=1,
                       layers_per_indexer=1, num_pages=4, num_idx_pages=4, max_requests=1, max_ctx=256, max_q_per_req=1,
                       hot_rows=64, max_tokens=1, idx_format=H.IDX_FP8, host_pages=1)
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        pool = H.Pool(cfg, [kv.data_ptr()], [idx.data_ptr()], host.data_ptr())
        assert pool.device is None
        pool.set_pages(0, 0, block_table=[2, 0], idx_pages=[1, 3], stream=0)
        assert pool.get_error(stream=0) == 0
    try:
        x = torch.randn(3, 576, device="cuda")
        req, pos = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.tensor([0, 1, 64], dtype=torch.int32, device="cuda")
        pool.append_quantized(0, req, pos, x[:, :512], x[:, 512:])
        assert pool.get_error() == 0 and pool.device == torch.cuda.current_device()
        want = CP.pack_rows(x[:, :512].cpu().numpy(), x[:, 512:].cpu().numpy())
        assert np.array_equal(kv[[128, 129, 0]].cpu().numpy(), want)
    finally:
        torch.cuda.synchronize()
        pool.close()
