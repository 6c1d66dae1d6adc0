"""A move of many pages is two launches, the check with its marks and then the copies. When the second one cannot be made,
no page is copied and no table changes, nor does a later move take the first one's marks for its own."""
import ctypes

import numpy as np
import pytest

from test_gpu_cache_ops import Cache, i32, torch
from test_gpu_pages import Model, moved, spare

pytestmark = pytest.mark.gpu


class FirstLaunch:
    """A call recorded as a graph from which every kernel but the first is taken out: what is left of the call on the
    device when its later launches fail on the host."""

    def __init__(self, call):
        self.cu = cu = ctypes.CDLL("libcuda.so.1")
        stream = torch.cuda.Stream()
        self.stream = ctypes.c_void_p(stream.cuda_stream)
        graph, execs, n = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_size_t(0)
        torch.cuda.synchronize()
        assert cu.cuStreamBeginCapture_v2(self.stream, 1) == 0        # of this thread
        call(stream.cuda_stream)
        assert cu.cuStreamEndCapture(self.stream, ctypes.byref(graph)) == 0
        assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
        self.kernels = n.value
        nodes, roots, one = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * 1)(), ctypes.c_size_t(1)
        assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
        assert cu.cuGraphGetRootNodes(graph, roots, ctypes.byref(one)) == 0 and one.value == 1
        for node in nodes:
            if node != roots[0]:
                assert cu.cuGraphDestroyNode(ctypes.c_void_p(node)) == 0
        assert cu.cuGraphInstantiateWithFlags(ctypes.byref(execs), graph, ctypes.c_ulonglong(0)) == 0
        self.graph, self.exec = graph, execs

    def launch(self):
        assert self.cu.cuGraphLaunch(self.exec, self.stream) == 0
        torch.cuda.synchronize()

    def close(self):
        torch.cuda.synchronize()
        assert self.cu.cuGraphExecDestroy(self.exec) == 0 and self.cu.cuGraphDestroy(self.graph) == 0


@pytest.mark.parametrize("before", [0, 1, 2])
def test_a_move_after_one_whose_copies_were_not_launched(before):
    n = 90
    with Cache(n_layers=2, lpi=1, pages=(n, n, 2), spare=n) as c:
        m = Model(c, 3)
        free, idx_free = spare(c)
        a, ia = np.array(c.table[0]), np.array(c.idx_table[0])
        b, ib = np.array(c.table[1]), np.array(c.idx_table[1])
        to, ito = np.array(free)[:n], np.array(idx_free)[:n]

        def move(src, dst, idx_src, idx_dst):
            c.pool.copy_pages(i32(src), i32(dst), i32(idx_src), i32(idx_dst), remap=True)
            moved(m, "kv", src, dst, True)
            moved(m, "idx", idx_src, idx_dst, True)
        for k in range(before):           # complete moves, there and back
            move(*((a, to, ia, ito) if k % 2 == 0 else (to, a, ito, ia)))
        home, ihome = (to, ito) if before % 2 else (a, ia)
        away, iaway = (a, ia) if before % 2 else (to, ito)
        ids = [i32(x) for x in (home, away, ihome, iaway)]
        half = FirstLaunch(lambda st: c.pool.copy_pages(*ids, remap=True, stream=st))
        assert half.kernels == 2
        half.launch()
        m.check()                         # neither pages nor tables
        # the other request's pages move: its entries alone follow
        move(b, away, ib, iaway)
        assert c.pool.get_error() == 0
        m.check()
        # twice more the half, with complete moves between and behind
        half.launch()
        half.launch()
        move(away, b, iaway, ib)
        m.check()
        move(home, away, ihome, iaway)
        assert c.pool.get_error() == 0
        m.check()
        half.close()
