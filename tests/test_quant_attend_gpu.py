"""Attention over a cache held in 4 or 8 bits against the fp64 definition on what
its rows stand for.

Tolerance per output element, u = 2^-24, N = 15 or 255, R = sum_r p_r |v_r| and R_w
the same sum of (n + z) s, which sums over codes are made of (L_w for logits):
- a logit is D products of codes summed in fp32 (the tensor cores drop bits toward
  zero, twice u per addition), the groups' zero codes taken off and the groups
  added up: |dx| <= 2 (D + 16) u L_w; where queries are held in fp16 beside their
  largest element q_top, each is within 2^-34 q_top: 2^-34 L_top; scaled: 4 u L_w;
- exponentials: ex2 is within 2^-22, its argument is rounded at |x| <= 2 L log2 e;
- sums over T rows, rescaled once per tile: 2 (T + 64) u R_w;
- on the tensor cores probabilities are rounded to fp16, alone and, for few rows, once
  more times the step: 2^-11 each of R_w (2^-10 is taken).  fp16 ends at 2^-24, half of
  which is lost per row: a probability of 1 stands at 2^6 or more, so T 2^-31 N S with
  the largest step S, and for few rows, at 2^11, T 2^-36 N S twice (codes and zero
  codes): together under T 2^-30 N S.  Steps below 2^-21 S lose bits: 2^-24 N S, twice;
- the output is rounded once: eps / 2 of its value.
lse moves by dx, the sum's T u and its own rounding."""
import math

import pytest
import torch

import quant_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def K():
    from eviction_kvc_score_gb300 import kvc
    return kvc


def rows_of(g, n, d, dt, strong):
    x = torch.randn((n, d), generator=g, device="cuda")
    if strong:
        x[:, ::41] = 3 * x[:, ::41] + 6
    return x.to(dt)


class Case:
    def __init__(self, ns, lens, hq, h, d, ps, dtype, bits, seed=0, gap=0, behind=0, spare=3, change=None):
        """ns: new tokens per sequence; lens: rows per list, new ones included;
        change(k, v): the lists' rows before they are written."""
        kvc = K()
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt, b = DT[dtype], len(ns)
        if len(lens) == b and not isinstance(lens[0], list):
            lens = [x for x in lens for _ in range(h)]
        lens = [x for row in lens for x in row] if isinstance(lens[0], list) else lens
        pages = [-(-x // ps) for x in lens]
        n_pages, width = sum(pages) + spare, max(pages) + 1
        self.lens, self.b, self.h, self.bits, self.dtype, self.scale = lens, b, h, bits, dtype, d ** -0.5
        self.max_new = max(max(ns), 1)
        self.c = kvc.cache(n_pages, ps, d, width, dtype)
        self.k = [rows_of(g, n, d, dt, True) for n in lens]
        self.v = [rows_of(g, n, d, dt, False) for n in lens]
        if change:
            change(self.k, self.v)
        size = kvc.kvc_quant_page_size(self.c, bits)
        # what lies behind a list may be anything: all ones is NaN in either format
        pools = [torch.randint(0, 256, (n_pages, size), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        pools[1][::2] = 255
        state = torch.empty(kvc.kvc_pages_size(self.c, b * h), dtype=torch.uint8, device="cuda")
        kvc.kvc_pages_init(self.c, state)
        table = torch.full((b * h, width), -1, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(b * h, dtype=torch.int32, device="cuda")
        n = torch.tensor(lens, device="cuda")
        src = [torch.cat(x + [torch.zeros((1, d), dtype=dt, device="cuda")]) for x in (self.k, self.v)]
        kvc.kvc_pages_append_quant(self.c, bits, table, self.len, n.int(), n.cumsum(0) - n, 1, *src, *pools, state)
        order = torch.randperm(n_pages, generator=g, device="cuda")
        self.kp, self.vp = (torch.empty_like(p) for p in pools)
        self.kp[order], self.vp[order] = pools[0], pools[1]
        self.table = torch.where(table >= 0, order[table.clamp(min=0).long()].int(), table)
        starts = [behind]
        for x in ns:
            starts.append(starts[-1] + x)
        self.start = starts
        n_tok = starts[-1] + behind
        buf = torch.randn((n_tok, hq * d + gap), generator=g, device="cuda").to(dt)
        self.q = buf[:, :hq * d].view(n_tok, hq, d)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(kvc.kvc_attend_quant_workspace_size(self.c, bits, hq, h, b, self.max_new), dtype=torch.uint8, device="cuda")
        kvc.kvc_workspace_init(self.ws)
        self.out = torch.full((n_tok, hq, d), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((n_tok, hq), 7.0, device="cuda")

    def run(self, **kw):
        a = dict(out=self.out, ws=self.ws, lse=self.lse, scale=self.scale)
        a.update(kw)
        K().kvc_attend_quant(self.c, self.bits, self.q, self.q_start, self.table, self.len, self.kp, self.vp, self.max_new, **a)
        return self

    def check(self, status=0, scale=None):
        torch.cuda.synchronize()
        assert K().kvc_workspace_status(self.ws) == status
        r = ref.attend(self.q, self.start, self.k, self.v, self.scale if scale is None else scale, self.bits)
        real = torch.zeros(self.lse.shape, dtype=torch.bool, device="cuda")
        real[self.start[0]:self.start[-1]] = True
        assert (self.out[~real] == 7).all() and (self.lse[~real] == 7).all()
        want, lse, d, t, n = r["out"], r["lse"], self.q.shape[-1], max(self.lens), ref.N[self.bits]
        dx = 2 * (d + 18) * U * r["logit_w"] + 2.0 ** -34 * r["logit_top"] + 2.0 ** -21
        tol = 2 * dx[..., None] * r["reach"] + 2 * (t + 64) * U * r["reach_w"]
        if self.dtype == "bf16" and d in (64, 128):
            tol = tol + 2.0 ** -10 * r["reach_w"] + (t * 2.0 ** -30 + 2.0 ** -23) * n * r["step"][..., None]
        tol = tol + want.abs() * torch.finfo(self.q.dtype).eps / 2 * 1.001
        fine = want.isfinite() & real[..., None]
        assert torch.equal(self.out.isnan() & real[..., None], want.isnan() & real[..., None])
        err = (self.out.double() - want).abs()
        bad = fine & ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), (err - tol)[fine].max().item(), torch.nonzero(bad)[:4].tolist())
        got, fine = self.lse.double(), lse.isfinite() & real
        assert torch.equal(got.isnan() & real, lse.isnan() & real)
        assert torch.equal(got[lse == -math.inf], lse[lse == -math.inf])
        tol = dx + 2 * (t + 64) * U + 4 * U * lse.abs()
        assert ((got - lse).abs() <= tol)[fine].all(), ((got - lse).abs() - tol)[fine].max()


CASES = [
    # one token
    dict(ns=[1], lens=[1], hq=4, h=4, d=64, ps=16),
    dict(ns=[1], lens=[1000], hq=32, h=8, d=128, ps=64),
    dict(ns=[1, 1, 1], lens=[[5, 700, 64], [128, 129, 1], [300, 17, 2049]], hq=12, h=3, d=128, ps=16),
    dict(ns=[1] * 7, lens=[127, 128, 129, 255, 256, 257, 4000], hq=8, h=2, d=64, ps=128),
    dict(ns=[1] * 9, lens=[15, 16, 17, 31, 32, 33, 63, 64, 65], hq=1, h=1, d=128, ps=16),
    dict(ns=[1, 0, 1], lens=[40, 30, 0], hq=2, h=1, d=64, ps=32),
    dict(ns=[1], lens=[9000], hq=71, h=1, d=64, ps=16),
    dict(ns=[1, 1], lens=[777, 778], hq=128, h=1, d=128, ps=64),
    dict(ns=[1], lens=[500], hq=130, h=1, d=128, ps=64),
    dict(ns=[1], lens=[100000], hq=4, h=1, d=128, ps=128),
    # a few tokens
    dict(ns=[5, 3], lens=[20000, 9000], hq=8, h=2, d=128, ps=64),
    dict(ns=[7, 1, 4], lens=[7, 1, 4], hq=6, h=2, d=64, ps=16),
    dict(ns=[8, 2, 1], lens=[700, 12, 90], hq=12, h=3, d=128, ps=32),
    dict(ns=[33], lens=[1500], hq=4, h=1, d=128, ps=32),
    dict(ns=[16, 31], lens=[16, 900], hq=8, h=1, d=128, ps=16),
    # chunks
    dict(ns=[200, 64, 129], lens=[200, 1000, 513], hq=4, h=2, d=128, ps=64),
    dict(ns=[300], lens=[300], hq=3, h=1, d=64, ps=16),
    dict(ns=[150, 90], lens=[700, 90], hq=5, h=1, d=128, ps=128),
    dict(ns=[257], lens=[2500], hq=2, h=2, d=128, ps=32),
    dict(ns=[65], lens=[4000], hq=7, h=1, d=128, ps=64),
    # chunks and single tokens in one call
    dict(ns=[180, 1, 1, 0, 1, 5], lens=[500, 100, 1, 9, 2222, 64], hq=8, h=2, d=128, ps=16),
    dict(ns=[1] * 40 + [150], lens=[33 * i + 1 for i in range(40)] + [1000], hq=4, h=1, d=64, ps=32),
    # lists shorter than the chunk: the first tokens see nothing
    dict(ns=[40, 10], lens=[[13, 40], [0, 3]], hq=4, h=2, d=128, ps=16),
    dict(ns=[6, 5], lens=[[3, 6], [0, 2]], hq=4, h=2, d=64, ps=16),
    dict(ns=[300], lens=[[100, 0]], hq=4, h=2, d=64, ps=64),
    # head sizes of the CUDA cores
    dict(ns=[3, 20], lens=[100, 333], hq=4, h=2, d=8, ps=16),
    dict(ns=[1, 40], lens=[999, 222], hq=6, h=3, d=80, ps=32),
    dict(ns=[2, 70], lens=[64, 300], hq=2, h=2, d=256, ps=128),
    dict(ns=[1, 19], lens=[100, 333], hq=4, h=2, d=192, ps=16),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_definition(i, dtype, bits):
    c = Case(**CASES[i], dtype=dtype, bits=bits, seed=i)
    c.run().check()
    again = c.out.clone(), c.lse.clone()
    c.out.fill_(7), c.lse.fill_(7)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, again[0]) and torch.equal(c.lse, again[1])


@pytest.mark.parametrize("bits,dtype,d,ns", [(4, "bf16", 128, [1, 1]), (8, "bf16", 64, [3, 90]), (4, "f32", 80, [2, 40])])
def test_strides_scale_and_tokens_of_no_sequence(bits, dtype, d, ns):
    c = Case(ns=ns, lens=[333, 500], hq=8, h=2, d=d, ps=32, dtype=dtype, bits=bits, gap=24, behind=5)
    c.run().check()
    for scale in (0.0, -0.3, 2.5):
        c.run(scale=scale).check(scale=scale)
    lse = c.lse.clone()
    c.run(lse=None, scale=2.5)
    c.check(scale=2.5)
    assert torch.equal(lse, c.lse)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d,ns", [("bf16", 128, [1, 1]), ("bf16", 128, [8, 3]), ("bf16", 64, [7, 1]), ("bf16", 128, [70, 40]),
                                        ("f32", 64, [5, 33]), ("bf16", 80, [1, 9])])
def test_nan_groups_reach_the_rows_that_see_them(ns, d, dtype, bits):
    """In K a row's logit is NaN, and all of its output; in V the group's channels."""
    def change(k, v):
        k[0][-1, 3] = math.inf          # seen by the last token alone
        k[1][100, 0] = math.nan
        v[2][-1, 40] = math.nan
        v[2][7, 1] = -math.inf
        v[3][-2, d - 1] = math.inf
        v[3][-1, 0] = 2.0 ** 126
    Case(ns=ns, lens=[[300, 200], [170, 90]], hq=4, h=2, d=d, ps=16, dtype=dtype, bits=bits, change=change).run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,ns", [("bf16", [1, 4]), ("bf16", [50, 33]), ("f32", [1, 9])])
def test_rows_of_very_different_sizes(ns, dtype, bits):
    """A few rows of V are thousands of times as large as the others, and a first
    row that takes most of the weight is small, as a cache's first rows are."""
    def change(k, v):
        for x in k:
            x[0] *= 8
        for x in v:
            x[0] *= 2.0 ** -7
            x[5::31] *= 2.0 ** 9
            x[7::50] *= 2.0 ** -12
            x[3::17, :32] = 0
    Case(ns=ns, lens=[900, 3000], hq=8, h=2, d=128, ps=64, dtype=dtype, bits=bits, change=change).run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d,n", [("bf16", 128, 1), ("bf16", 64, 6), ("bf16", 128, 60), ("f32", 96, 3)])
def test_large_logits(n, d, dtype, bits):
    """Softmaxes of one row, the maximum somewhere in the list."""
    def change(k, v):
        for i, x in enumerate(k):
            x.mul_(6)
            x[(i * 97 + 11) % x.shape[0]] *= 4
    c = Case(ns=[n, n], lens=[1000, 130], hq=6, h=2, d=d, ps=32, dtype=dtype, bits=bits, change=change)
    c.q.mul_(5)
    c.run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", [1, 5, 80])
def test_bad_pages_are_rows_of_zeros(n, bits):
    kvc = K()
    c = Case(ns=[n, n], lens=[200, 330], hq=4, h=2, d=128, ps=32, dtype="bf16", bits=bits)
    c.table[0, 2], c.table[1, 0], c.table[3, 9] = c.c.n_pages, -1, 2 ** 31 - 1
    for i, j in ((0, 2), (1, 0), (3, 9)):
        c.k[i][32 * j:32 * j + 32], c.v[i][32 * j:32 * j + 32] = 0, 0
    c.run().check(status=kvc.DEV_BAD_PAGE)


@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 40), ("f32", 2)])
def test_lengths_and_starts_out_of_range_are_cut(dtype, n):
    kvc = K()
    c = Case(ns=[n, n, n], lens=[90, 50, 33], hq=4, h=1, d=64, ps=16, dtype=dtype, bits=4)
    most = c.c.max_pages * 16
    c.len[2] = 2 ** 31 - 1     # as many rows as the table holds; its entries behind the list are -1
    zeros = [torch.zeros((most - 33, 64), dtype=DT[dtype], device="cuda") for _ in range(2)]
    # the rest of the list's last page keeps what lay there: cut it off
    c.table[2, 2] = -1
    c.k[2], c.v[2] = torch.cat([c.k[2][:32], zeros[0], c.k[2][:1] * 0]), torch.cat([c.v[2][:32], zeros[1], c.v[2][:1] * 0])
    c.lens[2] = most
    c.run().check(status=kvc.DEV_BAD_LIST | kvc.DEV_BAD_PAGE)


@pytest.mark.parametrize("bits", [4, 8])
def test_one_workspace_for_caches_of_every_kind(bits):
    """Calls of other types, sizes and kernels in between, on one workspace."""
    kvc = K()
    cases = [Case(ns=[1] * 9, lens=[40 * i + 7 for i in range(9)], hq=8, h=2, d=128, ps=16, dtype="bf16", bits=bits),
             Case(ns=[90, 1], lens=[900, 70], hq=8, h=2, d=64, ps=32, dtype="bf16", bits=12 - bits),
             Case(ns=[3, 20], lens=[30, 2000], hq=4, h=4, d=80, ps=64, dtype="f32", bits=bits)]
    ws = torch.empty(max(c.ws.numel() for c in cases), dtype=torch.uint8, device="cuda")
    kvc.kvc_workspace_init(ws)
    for c in cases:
        c.ws = ws
    for _ in range(3):
        for c in cases:
            c.out.fill_(7), c.lse.fill_(7)
            c.run()
    for c in cases:
        c.check()


def test_captured_graph_follows_new_lengths():
    kvc = K()
    c = Case(ns=[1] * 4, lens=[700, 30, 64, 3000], hq=8, h=2, d=128, ps=16, dtype="bf16", bits=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.run()
        for cut in (0, 29, 5):
            c.lens = [n - min(cut, n) for n in c.lens]
            c.k, c.v = [x[:n] for x, n in zip(c.k, c.lens)], [x[:n] for x, n in zip(c.v, c.lens)]
            c.len.copy_(torch.tensor(c.lens, dtype=torch.int32))
            graph.replay()
            side.synchronize()
            c.check()


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    a = Case(ns=[1] * 30, lens=[900 + i for i in range(30)], hq=8, h=2, d=128, ps=16, dtype="bf16", bits=4)
    b = Case(ns=[60, 1], lens=[1500, 8], hq=8, h=2, d=128, ps=32, dtype="bf16", bits=8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c in zip(streams, (a, b)):
            c.run(stream=s)
    a.check()
    b.check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 96), ("f32", 128)])
@pytest.mark.parametrize("ns", [[3, 1], [200, 64]])
def test_queries_that_are_no_numbers_spoil_their_own_rows(ns, dtype, d, bits):
    c = Case(ns=ns, lens=[700, 300], hq=6, h=2, d=d, ps=32, dtype=dtype, bits=bits, seed=d + bits)
    c.q[1, 2, 5] = math.nan
    c.q[2, 0, 3], c.q[2, 0, 40] = math.inf, -math.inf   # some key's two terms cancel
    c.run().check()
    assert c.out[1, 2].isnan().all() and c.out[2, 0].isnan().all() and int(c.out.isnan().any(-1).sum()) == 2


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 40), ("f32", 1), ("f32", 40)])
def test_pages_past_32_bits(n, dtype, bits):
    """Pages at the end of pools of more than 2^32 bytes."""
    kvc = K()
    c = Case(ns=[n], lens=[333], hq=4, h=2, d=128, ps=64, dtype=dtype, bits=bits)
    few, size = c.kp.shape
    c.c = kvc.cache(2 ** 32 // size + 1 + few, 64, 128, c.table.shape[1], dtype)
    move = c.c.n_pages - few
    pools = [torch.zeros((c.c.n_pages, size), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pools[0][move:], pools[1][move:] = c.kp, c.vp
    c.kp, c.vp = pools
    c.table = torch.where(c.table >= 0, c.table + move, c.table)
    c.run().check()


@pytest.mark.parametrize("ns,hq,h,d,dtype,bits", [
    ([1] * 40 + [30], 24, 1, 128, "bf16", 4),    # a token's 24 rows: two units of 16
    ([1] * 40 + [30], 24, 1, 64, "bf16", 8),
    ([1] * 130, 96, 4, 128, "bf16", 8),          # 520 lists of two units
    ([1] * 162 + [100], 32, 8, 64, "bf16", 4),   # 1,304 lists of up to two units, most of them another launch's
    ([1] * 129 + [100], 8, 4, 80, "f32", 8),     # 520 lists of up to four units
    ([3, 0] * 70 + [150], 8, 4, 128, "f32", 4),  # 564 lists of up to five
])
def test_many_lists_of_few_units(ns, hq, h, d, dtype, bits):
    lens = [n + 7 * i % 150 for i, n in enumerate(ns)]
    Case(ns=ns, lens=lens, hq=hq, h=h, d=d, ps=16, dtype=dtype, bits=bits, seed=d).run().check()
