"""The operators around a shared cache in a run of them as a server makes it: a prompt rotated and quantised
into the cache, forked into samples, decoded behind the shared prompt, its pages moved in between; eager,
captured and replayed, on two pools by two threads, and as the first calls of a process."""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

import cache_plain as CP
from test_gpu_cache_ops import Cache, check_chunk, i32, make_q, torch, values
from test_gpu_rotary import angles, check

pytestmark = pytest.mark.gpu
SM = 1 / math.sqrt(576)


class Server:
    """A prompt of n positions in request 0, and `samples` forks of it that decode a token at a time."""

    def __init__(self, heads=16, n=300, samples=12, seed=0, stream=None):
        from sparse_mla_kv_indexer_gb300 import hisparse as H
        self.n, self.samples, self.heads, self.stream = n, samples, heads, stream
        pages = -(-n // 64)
        self.c = c = Cache(heads=heads, n_layers=2, lpi=2, pages=(pages,) + (1,) * samples, max_ctx=-(-(n + 8) // 128) * 128,
                           spare=pages + samples, seed=seed)
        for r in range(samples):      # the forks begin with nothing of their own
            c.pool.set_pages(r + 1, 0, block_table=[-1], idx_pages=[-1])
        self.tails = [int(c.table[r + 1][0]) for r in range(samples)]
        self.idx_tails = [int(c.idx_table[r + 1][0]) for r in range(samples)]
        self.rng = np.random.default_rng(seed)
        steps, self.magnitude = H.rotary_steps(64, 10000.0, "ramp", factor=8.0, original_ctx=128.0, magnitude=0.1)
        self.host_steps, self.steps = steps, steps.cuda()
        self.kv = [np.zeros((0, 576))] * (samples + 1)
        k = samples
        self.req, self.pos, self.limit = i32(range(1, k + 1)), i32([n] * k), i32([n + 1] * k)
        self.seg_start, self.groups, self.length = i32(range(k + 1)), i32([0, k]), i32([n])
        self.lat, self.raw = torch.zeros(k, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(k, 64, dtype=torch.bfloat16, device="cuda")
        self.rope = torch.zeros_like(self.raw)
        self.keys = torch.zeros(k, 128, dtype=torch.bfloat16, device="cuda")
        self.up = torch.zeros(k, heads, 192, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(k, heads, 576, dtype=torch.bfloat16, device="cuda")
        self.out, self.lse = torch.zeros(k, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(k, heads, device="cuda")
        self.work = torch.empty(c.pool.prefix_workspace_bytes(k, k, 1), dtype=torch.uint8, device="cuda")

    def begin(self):
        """The prompt, then the forks."""
        c, n, k = self.c, self.n, self.samples
        lat, lf = values(self.rng, n, 512, "bf16", 0.3)
        raw, _ = values(self.rng, n, 64, "bf16", 0.3)
        keys, kf = values(self.rng, n, 128, "bf16", 0.3)
        rope, every = torch.empty_like(raw), i32(range(n))
        p, s = c.pool, self.stream
        torch.cuda.synchronize()
        p.rotary(every, self.steps, [(raw, rope, "pairs")], magnitude=self.magnitude, stream=s)
        p.append_quantized(1, i32([0] * n), every, lat, rope, keys, stream=s)
        p.fork_requests(i32([0] * k), i32(range(1, k + 1)), i32([n] * k), i32(self.tails), i32(self.idx_tails), stream=s)
        torch.cuda.synchronize()
        check(rope, raw, angles(range(n), self.host_steps), "pairs", "bf16", self.magnitude)
        rows = CP.pack_rows(lf, rope.float().cpu().numpy())
        self.kv = [CP.row_values(rows)] * (k + 1)
        self.prompt_keys = CP.quantise(kf)

    def inputs(self, step):
        k = self.samples
        for t, width in ((self.lat, 512), (self.raw, 64), (self.keys, 128)):
            t.copy_(values(self.rng, k, width, "bf16", 0.3)[0])
        x = make_q(self.rng, k, self.heads, "bf16")
        self.q[:, :, :512].copy_(x[:, :, :512])
        self.up[:, :, 128:].copy_(x[:, :, 512:])
        self.pos.fill_(self.n + step)
        self.limit.fill_(self.n + step + 1)
        torch.cuda.synchronize()

    def decode(self, stream=None):
        p, s = self.c.pool, stream or self.stream
        p.rotary(self.pos, self.steps, [(self.up[:, :, 128:], self.q[:, :, 512:], "pairs"), (self.raw, self.rope, "pairs")],
                 magnitude=self.magnitude, stream=s)
        p.append_quantized(1, self.req, self.pos, self.lat, self.rope, self.keys, stream=s)
        p.prefix_attention(1, self.groups, self.length, self.req, self.seg_start, self.limit, self.q, SM, self.out, self.work,
                           lse=self.lse, stream=s)

    def check(self, step):
        torch.cuda.synchronize()
        assert self.c.pool.get_error() == 0
        w = angles([self.n + step] * self.samples, self.host_steps)
        check(self.rope, self.raw, w, "pairs", "bf16", self.magnitude)
        check(self.q[:, :, 512:], self.up[:, :, 128:], w, "pairs", "bf16", self.magnitude)
        rows = CP.row_values(CP.pack_rows(self.lat.float().cpu().numpy(), self.rope.float().cpu().numpy()))
        self.kv = self.kv[:1] + [np.r_[self.kv[r + 1], rows[r:r + 1]] for r in range(self.samples)]
        check_chunk(self.c, self.kv, range(1, self.samples + 1), range(self.samples + 1), [self.n + step + 1] * self.samples, self.q, SM,
                    self.out, self.lse, "bf16")

    def move(self, back=False):
        """Half of the prompt's pages and half of the tails to pages that nothing names (or back), in both caches."""
        c, k = self.c, self.samples
        some = [int(x) for x in c.table[0][::2]] + self.tails[::2]
        some_idx = [int(x) for x in c.idx_table[0][::2]] + self.idx_tails[::2]
        used = {int(x) for t in c.table for x in t}, {int(x) for t in c.idx_table for x in t}
        free = [[p for p in range(c.n_pages) if p not in u] for u in used]
        to, to_idx = free[0][:len(some)], free[1][:len(some_idx)]
        a, b = (some, some_idx), (to, to_idx)
        if back:
            a, b = b, a
        return [i32(a[0]), i32(b[0]), i32(a[1]), i32(b[1])]


@pytest.mark.parametrize("heads,n", [(16, 300), (64, 1025)])
def test_prompt_fork_decode_and_move(heads, n):
    s = Server(heads, n)
    with s.c as c:
        s.begin()
        for step in range(4):
            s.inputs(step)
            if step == 2:
                moves = s.move()
                c.pool.copy_pages(*moves, remap=True)
                torch.cuda.synchronize()
                for layer in c.kv:        # what is left behind is free
                    layer.view(-1, 64, 656)[moves[0].long()] = 255
                for idx in c.idx:
                    idx[moves[2].long()] = 255
            s.decode()
            s.check(step)
        # the prompt's keys, read through a fork's tables after the move
        keys = torch.empty(n, 128, device="cuda")
        c.pool.read_rows(1, i32([3] * n), i32(range(n)), keys=keys)
        codes, scale = s.prompt_keys
        want = CP.e4m3_to_f64(codes) * scale.astype(np.float64)
        assert np.array_equal(keys.cpu().numpy(), want.astype(np.float32)) and c.pool.get_error() == 0


def test_captured_steps_and_moves_replayed():
    """A decode step, a move and the move back in three graphs on one stream, which share the workspace, replayed
    with other inputs; forks again from a graph."""
    s = Server(seed=1)
    with s.c as c:
        k = s.samples
        there, back = s.move(), s.move(back=True)
        forks = [i32([0] * k), i32(range(1, k + 1)), i32([s.n] * k), i32(s.tails), i32(s.idx_tails)]
        table = torch.zeros(k + 1, c.max_ctx // 64, dtype=torch.int32, device="cuda")
        every = i32(range(k + 1))
        torch.cuda.synchronize()
        graphs = [torch.cuda.CUDAGraph() for _ in range(4)]
        calls = [s.decode, lambda: c.pool.copy_pages(*there, remap=True),
                 lambda: c.pool.copy_pages(*back, remap=True),
                 lambda: (c.pool.fork_requests(*forks), c.pool.get_pages(every, 0, table))]
        for g, call in zip(graphs, calls):
            with torch.cuda.graph(g):
                call()
        s.begin()
        step, move, home, fork = graphs
        at = 0
        for g in (None, move, home, move, home):
            if g is not None:
                g.replay()
            s.inputs(at)
            step.replay()
            s.check(at)
            at += 1
        # every fork begins again: what the samples had appended is gone
        fork.replay()
        assert np.array_equal(table[1:, :s.n // 64].cpu().numpy(), np.tile(c.table[0][:s.n // 64], (k, 1)))
        s.kv = [v[:s.n] for v in s.kv]
        s.inputs(0)
        step.replay()
        s.check(0)


def test_two_threads_two_pools_two_streams():
    sides = [Server(16, 200, 6, seed=2, stream=torch.cuda.Stream()), Server(32, 333, 10, seed=3, stream=torch.cuda.Stream())]
    with sides[0].c, sides[1].c:
        for s in sides:
            s.begin()
            s.inputs(0)
        failed = []

        def work(s):
            try:
                for _ in range(30):
                    s.decode()
            except Exception as e:       # a thread's own exception would be lost
                failed.append(e)
        threads = [threading.Thread(target=work, args=(s,)) for s in sides]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed
        for s in sides:
            s.check(0)


FIRST = """
import os, sys
sys.path[:0] = [os.getcwd(), os.path.join(os.getcwd(), "tests")]
import torch
from test_gpu_shared_chain import Server
s = Server(seed=5)
with s.c as c:
    moves = s.move()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.pool.copy_pages(*moves, remap=True)
        s.decode()
    s.begin()
    s.inputs(0)
    g.replay()
    s.check(0)
print("captured")
"""


def test_the_first_calls_of_a_process_are_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
