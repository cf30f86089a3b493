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


class Many:
    """2^20 lists of no rows, a token of every sequence, and more units of max_new tokens than can be counted."""
    def __init__(self, dtype, d, heads, max_new):
        kvc, dt = K(), dict(f32=torch.float32, bf16=torch.bfloat16)[dtype]
        self.c, self.heads, self.max_new, seqs = kvc.cache(4, 16, d, 1, dtype), heads, max_new, 1 << 17
        empty = lambda *x, **kw: torch.empty(*x, device="cuda", **kw)  # noqa: E731
        self.q = torch.zeros((1, heads, d), dtype=dt, device="cuda").expand(seqs, heads, d)
        self.q_start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
        self.table, self.lens = torch.zeros((8 * seqs, 1), dtype=torch.int32, device="cuda"), torch.zeros(8 * seqs, dtype=torch.int32, device="cuda")
        self.out = torch.full((seqs, heads, d), 7.0, dtype=dt, device="cuda")
        self.q = self.q.contiguous()
        self.pool = empty(4 * 16 * d * 4, dtype=torch.uint8)
        self.ws = empty(kvc.kvc_attend_quant_workspace_size(self.c, 4, heads, 8, seqs, max_new), dtype=torch.uint8)
        kvc.kvc_workspace_init(self.ws)

    def quant(self, bits):
        pool = self.pool[:4 * K().kvc_quant_page_size(self.c, bits)]
        K().kvc_attend_quant(self.c, bits, self.q, self.q_start, self.table, self.lens, pool, pool, self.max_new, self.out, self.ws)

    def plain(self):
        pool = self.pool.view(self.q.dtype)[:4 * 16 * self.q.shape[-1]]
        K().kvc_attend(self.c, self.q, self.q_start, self.table, self.lens, pool, pool, self.max_new, self.out, self.ws)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 80), ("f32", 64)])
def test_refused_launches_name_the_call(dtype, d):
    m = Many(dtype, d, 8, 1 << 22)
    for bits in (4, 8):
        with pytest.raises(K().KvcError, match="kvc_attend_quant: n_seqs . n_kv_heads . max_new is too large"):
            m.quant(bits)
    with pytest.raises(K().KvcError, match="kvc_attend: n_seqs . n_kv_heads . max_new is too large"):
        m.plain()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 80), ("f32", 64)])
def test_refused_launches_write_nothing(dtype, d):
    m = Many(dtype, d, 8, 1 << 22)
    for bits in (4, 8):
        with pytest.raises(K().KvcError):
            m.quant(bits)
    torch.cuda.synchronize()
    assert (m.out == 7).all()
