"""Which kernels a call of kvc_attend_quant launches, and what its launches refuse."""
import ctypes as C

import pytest
import torch

from test_quant_attend_gpu import Case, K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def launches(call):
    """Kernels of a call, counted as the nodes of a graph that it is captured into."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = C.c_size_t(0)
    assert C.CDLL("libcuda.so.1").cuGraphGetNodes(C.c_void_p(graph.raw_cuda_graph()), None, C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("ns,hq,h,d,want", [
    ([1, 1, 1], 8, 2, 128, 1),        # a token each
    ([1, 1, 1], 64, 1, 128, 1),       # 64 query heads per KV head: more rows than the kernel of few takes
    ([1, 1], 71, 1, 64, 1),
    ([1, 1], 256, 2, 128, 1),
    ([1, 1], 66, 2, 64, 1),
    ([1, 1], 64, 2, 64, 1),           # 32
    ([1, 1, 20], 64, 2, 64, 1),       # and a chunk beside them: 235 rows a list, more than 128
    ([1] * 9 + [20], 64, 2, 64, 2),   # 93
    ([1, 1, 1, 40], 8, 2, 128, 2),
    ([90, 80], 8, 2, 128, 1),         # chunks alone
])
def test_no_launch_that_has_nothing_to_do(ns, hq, h, d, want, bits):
    c = Case(ns=ns, lens=[100 + n for n in ns], hq=hq, h=h, d=d, ps=16, dtype="bf16", bits=bits)
    assert launches(c.run) == want
    c.check()
