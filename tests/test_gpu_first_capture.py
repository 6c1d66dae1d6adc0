"""The cache operators captured into a graph by the first calls that a process makes of them, and
replayed; two threads that call two pools at once."""
import subprocess
import sys
import threading

import numpy as np
import pytest

import cache_plain as CP
from test_gpu_cache_ops import Cache, check_chunk, i32, make_q, torch, values

pytestmark = pytest.mark.gpu

FIRST = """
import os, sys
sys.path[:0] = [os.getcwd(), os.path.join(os.getcwd(), "tests")]
import numpy as np, torch
import cache_plain as CP
from test_gpu_cache_ops import Cache, check_chunk, i32, make_q, values
rng = np.random.default_rng(0)
for dtype in ("bf16", "fp16"):
    with Cache(heads=16, n_layers=1, lpi=1, pages=(3,)) as c:
        n = 150
        lat, lf = values(rng, n, 512, dtype, 0.3)
        rope, rf = values(rng, n, 64, dtype, 0.3)
        q = make_q(rng, n, 16, dtype)
        out, lse = torch.zeros(n, 16, 512, dtype=q.dtype, device="cuda"), torch.zeros(n, 16, device="cuda")
        back = torch.zeros(n, 512, dtype=q.dtype, device="cuda")
        req, pos, lim, sr, ss = i32([0] * n), i32(range(n)), i32(range(1, n + 1)), i32([0]), i32([0, n])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.pool.append_quantized(0, req, pos, lat, rope)
            c.pool.chunk_attention(0, sr, ss, lim, q, 1 / 24, out, c.work, lse=lse)
            c.pool.read_rows(0, req, pos, back)
        g.replay()
        torch.cuda.synchronize()
        assert c.pool.get_error() == 0
        rows = CP.pack_rows(lf, rf)
        assert np.array_equal(c.get_rows(0, 0, np.arange(n)), rows)
        kv = CP.row_values(rows)
        check_chunk(c, [kv], [0], [0, n], np.arange(1, n + 1), q, 1 / 24, out, lse, dtype, set(range(0, n, 7)))
        assert torch.equal(back.cpu(), torch.from_numpy(kv[:, :512].astype(np.float32)).to(q.dtype))
print("captured")
"""


def test_the_first_calls_of_a_process_are_captured():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_two_threads_call_two_pools():
    """Each thread appends, attends and reads back on its own stream, pool and workspace."""
    sides = []
    with Cache(heads=16, n_layers=1, lpi=1, pages=(5,), seed=3) as a, Cache(heads=64, n_layers=1, lpi=1, pages=(5,), seed=4) as b:
        for k, c in enumerate((a, b)):
            rng = np.random.default_rng(k)
            n = 300
            lat, lf = values(rng, n, 512, "bf16", 0.3)
            rope, rf = values(rng, n, 64, "bf16", 0.3)
            q = make_q(rng, 20, c.heads, "bf16")
            sides.append(dict(c=c, n=n, lat=lat, rope=rope, rows=CP.pack_rows(lf, rf), q=q, stream=torch.cuda.Stream(),
                              out=torch.zeros(20, c.heads, 512, dtype=torch.bfloat16, device="cuda"),
                              lse=torch.zeros(20, c.heads, device="cuda"), back=torch.zeros(n, 512, device="cuda"),
                              req=i32([0] * n), pos=i32(range(n)), lim=i32(range(281, 301)), sr=i32([0]), ss=i32([0, 20])))
        torch.cuda.synchronize()
        failed = []

        def work(s):
            try:
                p = s["c"].pool
                for _ in range(30):
                    p.append_quantized(0, s["req"], s["pos"], s["lat"], s["rope"], stream=s["stream"])
                    p.chunk_attention(0, s["sr"], s["ss"], s["lim"], s["q"], 1 / 24, s["out"], s["c"].work, lse=s["lse"],
                                      stream=s["stream"])
                    p.read_rows(0, s["req"], s["pos"], s["back"], stream=s["stream"])
            except Exception as e:                     # a thread's own exception would be lost
                failed.append(e)
        threads = [threading.Thread(target=work, args=(s,)) for s in sides]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed
        for s in sides:
            c, kv = s["c"], CP.row_values(s["rows"])
            assert c.pool.get_error() == 0
            assert np.array_equal(c.get_rows(0, 0, np.arange(s["n"])), s["rows"])
            assert np.array_equal(s["back"].cpu().numpy(), kv[:, :512].astype(np.float32))
            check_chunk(c, [kv], [0], [0, 20], np.arange(281, 301), s["q"], 1 / 24, s["out"], s["lse"], "bf16")
