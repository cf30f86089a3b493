"""Attention over the paged cache against the fp64 definition.

Tolerance per output element, u = 2^-24 and reach R = sum_r p_r |v_r|:
- a logit is D products summed in fp32 (the tensor cores drop bits toward zero,
  twice u per addition) and scaled: |dx| <= 2 (D + 4) u L, L the row's largest
  sum_d |q_d k_d| scale; numerator and denominator each move by that;
- exponentials: ex2 is within 2^-22, its argument is rounded at |x| <= 2 L log2 e;
- sums over T rows, rescaled once per tile: 2 (T + 64) u R;
- on the tensor cores each probability is rounded to bf16: 2^-8 R;
- the output is rounded once: eps / 2 of its value.
lse moves by dx, the sum's T u and its own rounding."""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu


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


DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


class Case:
    def __init__(self, ns, lens, hq, h, d, ps, dtype, seed=0, gap=0, behind=0, spare=3, junk=math.nan):
        """ns: new tokens per sequence; lens: rows per list, new ones included."""
        kvc = K()
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = DT[dtype]
        b = len(ns)
        if len(lens) == b:
            lens = [x for x in lens for _ in range(h)]
        pages = [-(-x // ps) for x in lens]
        n_pages, width = sum(pages) + spare, max(pages) + 1
        self.lens, self.ns, self.b, self.h = lens, ns, b, h
        self.max_new = max(max(ns), 1)
        self.c = kvc.cache(n_pages, ps, d, width, dtype)
        self.kp = torch.randn((n_pages, ps, d), generator=g, device="cuda").to(dt)
        self.vp = torch.randn((n_pages, ps, d), generator=g, device="cuda").to(dt)
        order = torch.randperm(n_pages, generator=g, device="cuda").int()
        self.table = torch.full((b * h, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, x in enumerate(lens):
            self.table[i, :pages[i]] = order[at:at + pages[i]]
            at += pages[i]
            if x % ps:   # what lies behind a list may be anything
                last = order[at - 1].item()
                self.kp[last, x % ps:] = junk
                self.vp[last, x % ps:] = junk
        self.len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [behind]
        for n in ns:
            starts.append(starts[-1] + n)
        self.start = starts
        n_tok = starts[-1] + behind
        buf = torch.randn((n_tok, hq * d + gap), generator=g, device="cuda").to(dt)
        self.q = buf[:, :hq * d].view(n_tok, hq, d)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(kvc.kvc_attend_workspace_size(self.c, hq, h, b, self.max_new), dtype=torch.uint8, device="cuda")
        kvc.kvc_workspace_init(self.ws)
        self.out = torch.full((n_tok, hq, d), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((n_tok, hq), 7.0, device="cuda")
        self.dtype, self.scale = dtype, d ** -0.5

    def run(self, **kw):
        a = dict(out=self.out, ws=self.ws, lse=self.lse, scale=self.scale)
        a.update(kw)
        K().kvc_attend(self.c, self.q, self.q_start, self.table, self.len, self.kp, self.vp, self.max_new, **a)
        return self

    def check(self, status=0):
        torch.cuda.synchronize()
        assert K().kvc_workspace_status(self.ws) == status
        want, lse, reach, logit = ref.attend(self.q, self.start, self.table, self.lens, self.kp, self.vp, self.scale)
        real = ~want.isnan()
        assert (self.out[~real] == 7).all() and (self.lse[~real[..., 0]] == 7).all()
        d = self.q.shape[-1]
        t = max(self.lens)
        dx = 2 * (d + 4) * U * logit + 4 * U * logit + 2.0 ** -21
        tc = self.dtype == "bf16" and d in (64, 128)
        tol = (2 * dx + 2 * (t + 64) * U + (2.0 ** -8 if tc else 0))[..., None] * reach + want.abs() * torch.finfo(self.q.dtype).eps / 2 * 1.001
        err = (self.out.double() - want).abs()
        bad = real & ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), (err - tol)[real].max().item(), torch.nonzero(bad)[:4].tolist())
        got, fine = self.lse.double(), lse.isfinite()
        assert torch.equal(got[lse == -math.inf], lse[lse == -math.inf])
        tol = dx + 2 * (t + 64) * U + 4 * U * lse.abs()
        assert ((got - lse).abs() <= tol)[fine].all(), ((got - lse).abs() - tol)[fine].max()


CASES = [
    # one token
    dict(ns=[1], lens=[1], hq=4, h=4, d=64, ps=16),
    dict(ns=[1], lens=[1000], hq=32, h=8, d=128, ps=64),
    dict(ns=[1, 1, 1], lens=[[5, 700, 64], [128, 129, 1], [300, 17, 2049]], hq=12, h=3, d=128, ps=16),
    dict(ns=[1] * 7, lens=[127, 128, 129, 255, 256, 257, 4000], hq=8, h=2, d=64, ps=128),
    dict(ns=[1, 0, 1], lens=[40, 30, 0], hq=2, h=1, d=64, ps=32),
    dict(ns=[1], lens=[9000], hq=71, h=1, d=64, ps=16),
    dict(ns=[1, 1], lens=[777, 778], hq=128, h=1, d=128, ps=64),
    dict(ns=[1], lens=[500], hq=130, h=1, d=128, ps=64),
    # a few tokens
    dict(ns=[5, 3], lens=[20000, 9000], hq=8, h=2, d=128, ps=64),
    dict(ns=[7, 1, 4], lens=[7, 1, 4], hq=6, h=2, d=64, ps=16),
    dict(ns=[33], lens=[1500], hq=4, h=1, d=128, ps=32),
    dict(ns=[16, 31], lens=[16, 900], hq=8, h=1, d=128, ps=16),
    # chunks
    dict(ns=[200, 64, 129], lens=[200, 1000, 513], hq=4, h=2, d=128, ps=64),
    dict(ns=[300], lens=[300], hq=3, h=1, d=64, ps=16),
    dict(ns=[150, 90], lens=[700, 90], hq=5, h=1, d=128, ps=128),
    dict(ns=[257], lens=[2500], hq=2, h=2, d=128, ps=32),
    dict(ns=[65], lens=[4000], hq=7, h=1, d=128, ps=64),
    # lists shorter than the chunk: the first tokens see nothing
    dict(ns=[40, 10], lens=[[13, 40], [0, 3]], hq=4, h=2, d=128, ps=16),
    dict(ns=[300], lens=[[100, 0]], hq=4, h=2, d=64, ps=64),
    # head sizes of the CUDA cores
    dict(ns=[3, 20], lens=[100, 333], hq=4, h=2, d=8, ps=16),
    dict(ns=[1, 40], lens=[999, 222], hq=6, h=3, d=80, ps=32),
    dict(ns=[2, 70], lens=[64, 300], hq=2, h=2, d=256, ps=128),
]


def flat(lens):
    return [x for row in lens for x in row] if isinstance(lens[0], list) else lens


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_the_definition(i, dtype):
    c = dict(CASES[i])
    c["lens"] = flat(c["lens"])
    Case(**c, dtype=dtype, seed=i, gap=8 * (i % 3), behind=i % 2 * 3).run().check()


@pytest.mark.parametrize("dtype,d,hq,h", [("f32", 64, 8, 2), ("f32", 80, 17, 1), ("bf16", 64, 8, 2), ("bf16", 128, 8, 2),
                                          ("bf16", 96, 6, 2)])
@pytest.mark.parametrize("ns", [[40, 1, 0, 3, 1, 17], [1, 1, 130, 5, 1], [4, 0, 5, 300]])
def test_chunks_and_single_tokens_in_one_call(dtype, d, hq, h, ns):
    lens = [900, 333, 60, 77, 1, 450][:len(ns)]
    Case(ns=ns, lens=lens, hq=hq, h=h, d=d, ps=32, dtype=dtype, seed=len(ns)).run().check()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 80)])
@pytest.mark.parametrize("ns", [[300] + [1] * 200 + [0] * 40 + [70, 2], [1, 0] * 60 + [1100] + [130, 0, 3] * 20])
def test_large_batches_of_chunks_and_single_tokens(dtype, d, ns):
    lens = [n + (37 * i % 700) * (n > 0 or i % 3 == 0) for i, n in enumerate(ns)]
    Case(ns=ns, lens=lens, hq=8, h=2, d=d, ps=32, dtype=dtype, seed=3).run().check()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("places,n", [(33, 1), (700, 1), (700, 20)])
def test_batches_whose_places_are_mostly_empty(dtype, d, places, n):
    """Few sequences have tokens; the others' lists are empty or keep their rows."""
    ns, lens = [0] * places, [(0, 40)[i % 2] for i in range(places)]
    for i in (1, places // 2, places - 1):
        ns[i], lens[i] = n, 300 + i % 7
    Case(ns=ns, lens=lens, hq=4, h=2, d=d, ps=16, dtype=dtype, seed=places).run().check()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 80)])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_rows_that_a_token_does_not_see_may_hold_anything(dtype, d, junk):
    """The last tokens' rows are NaN or infinite: earlier tokens' outputs do not change by a bit."""
    c = Case(ns=[40, 3], lens=[140, 260], hq=4, h=2, d=d, ps=16, dtype=dtype, seed=5, junk=junk).run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    for s in range(2):
        for h in range(2):
            i = s * 2 + h
            for r in range(c.lens[i] - (10, 1)[s], c.lens[i]):
                page = c.table[i, r // 16].item()
                c.kp[page, r % 16] = junk
                c.vp[page, r % 16] = junk
    c.run()
    torch.cuda.synchronize()
    kept = [*range(30), 40, 41]
    assert torch.equal(c.out[kept], out[kept]) and torch.equal(c.lse[kept], lse[kept])
    assert not c.out[[39, 42]].isfinite().any()


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_that_are_seen_reach_the_outputs(d):
    """One infinite element of a row near the diagonal: the tokens that see it get it, in that column alone."""
    c = Case(ns=[40], lens=[140], hq=4, h=2, d=d, ps=16, dtype="bf16", seed=6)
    page = c.table[0, 130 // 16].item()
    c.vp[page, 130 % 16, 3] = math.inf
    c.run()
    torch.cuda.synchronize()
    assert (c.out[30:, :2, 3] == math.inf).all()
    c.out[30:, :2, 3] = 0
    assert c.out.isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_logit_is_too_large_or_too_small(dtype):
    c = Case(ns=[1, 30], lens=[900, 500], hq=4, h=2, d=128, ps=64, dtype=dtype, seed=7)
    c.scale = 20.0          # one row takes it all, far from the first
    c.run().check()
    c.scale = -3.0
    c.run().check()
    c.scale = 0.0           # the plain mean
    c.run().check()
    c.kp.mul_(1e4)
    c.kp.nan_to_num_(nan=math.nan)
    c.scale = 1e-4
    c.run().check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_row_whose_logits_are_all_minus_infinity(dtype):
    """That is a softmax of nothing but -infinity, as in the formula: NaN; not the zeros of a row that sees nothing."""
    c = Case(ns=[1, 1], lens=[300, 200], hq=2, h=1, d=64, ps=16, dtype=dtype, seed=8)
    c.q[0, 0] = 1.0
    for r in range(300):
        c.kp[c.table[0, r // 16].item(), r % 16] = -math.inf
    c.run()
    torch.cuda.synchronize()
    assert c.out[0, 0].isnan().all() and c.out[1].isfinite().all()


@pytest.mark.parametrize("dtype,case", [("f32", 8), ("bf16", 8), ("bf16", 12), ("bf16", 5)])
def test_same_bits_again_and_from_a_graph(dtype, case):
    c = Case(**{**CASES[case], "lens": flat(CASES[case]["lens"])}, dtype=dtype, seed=9).run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run()
        c.run()      # two calls of one graph share the workspace
    for _ in range(5):
        c.out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    # new lengths are read on the device: the graph goes on with them
    c.lens = [max(0, x - 1) for x in c.lens]
    c.len.copy_(torch.tensor(c.lens, dtype=torch.int32))
    graph.replay()
    c.check()


@pytest.mark.parametrize("dtype,d,hq", [("f32", 64, 2), ("bf16", 64, 2), ("bf16", 128, 40), ("bf16", 96, 2)])
def test_neighbouring_lists_that_fill_the_gpu(dtype, d, hq):
    """Two long lists share one block of the launch, at every place of its work: the joins of
    the first list's end and of the second one's beginning do not meet."""
    c = Case(ns=[1, 1], lens=[40000, 40000], hq=hq, h=1, d=d, ps=128, dtype=dtype, seed=8)
    for cut in range(0, 12000, 192):
        c.lens = [40000 - cut, 40000]
        c.len.copy_(torch.tensor(c.lens, dtype=torch.int32))
        for again in range(4):
            c.out.fill_(7)
            c.run()
            out = c.out.clone() if again == 0 else out
            assert torch.equal(c.out, out), (cut, again)
        c.check()


def test_two_streams_with_workspaces_of_their_own():
    a = Case(ns=[5, 3], lens=[20000, 9000], hq=8, h=2, d=128, ps=64, dtype="bf16", seed=10)
    b = Case(ns=[200], lens=[3000], hq=8, h=2, d=64, ps=16, dtype="bf16", seed=11)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a.run(stream=s)
        b.run(stream=t)
    a.check()
    b.check()


def test_one_workspace_serves_caches_of_several_kinds():
    cases = [Case(ns=[5, 3], lens=[20000, 9000], hq=8, h=2, d=128, ps=64, dtype="bf16", seed=20),
             Case(ns=[1, 2], lens=[9000, 700], hq=8, h=2, d=64, ps=64, dtype="f32", seed=21),
             Case(ns=[40], lens=[3000], hq=8, h=1, d=80, ps=16, dtype="bf16", seed=22),
             Case(ns=[300], lens=[3000], hq=8, h=1, d=64, ps=16, dtype="bf16", seed=23)]
    ws = max((c.ws for c in cases), key=lambda w: w.numel())
    for _ in range(2):
        for c in cases:
            c.ws = ws
            c.run().check()


def test_lists_that_share_pages():
    """Forked lists: the same pages in several rows of the table."""
    c = Case(ns=[1, 1, 1], lens=[500, 500, 500], hq=4, h=2, d=128, ps=64, dtype="bf16", seed=24)
    c.table[2:4] = c.table[0:2]
    c.table[4:6] = c.table[0:2]
    c.q[1:] = c.q[0]
    c.run().check()
    assert torch.equal(c.out[1], c.out[0]) and torch.equal(c.out[2], c.out[0])


def test_bad_pages_count_as_rows_of_zeros():
    for d, dtype in ((128, "bf16"), (64, "f32")):
        c = Case(ns=[1, 20], lens=[200, 100], hq=2, h=1, d=d, ps=16, dtype=dtype, seed=12)
        good = c.table.clone()
        for bad in (-1, c.c.n_pages, 1 << 30, -(1 << 31)):
            c.table[0, 3] = bad
            c.run()
            # the definition reads a page of zeros there instead
            zero = c.c.n_pages - 1
            while (good == zero).any():
                zero -= 1
            c.kp[zero], c.vp[zero] = 0, 0
            c.table[0, 3] = zero
            c.check(status=0x40)
            K().kvc_workspace_init(c.ws)


def test_bad_lengths_are_cut():
    c = Case(ns=[1, 2], lens=[100, 64], hq=2, h=1, d=64, ps=16, dtype="bf16", seed=13)
    c.len[0] = -3
    c.len[1] = 1 << 30
    c.table[1] = c.table[1, :1]      # every entry a page of the pool
    c.run()
    torch.cuda.synchronize()
    assert K().kvc_workspace_status(c.ws) == 0x20
    assert (c.out[0] == 0).all() and (c.lse[0] == -math.inf).all()
    # q_start outside the tokens, backwards, longer than max_new
    for starts in ([-5, 2, 3], [0, 2, 1], [0, 1, 9], [0, 3, 3]):
        c = Case(ns=[1, 2], lens=[100, 64], hq=2, h=1, d=64, ps=16, dtype="bf16", seed=13)
        c.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
        c.run()
        torch.cuda.synchronize()
        assert K().kvc_workspace_status(c.ws) == 0x20, starts


def test_pools_beyond_32_bit_offsets():
    """Rows past 2^31 elements of a pool."""
    kvc, d, ps, n_pages = K(), 128, 128, (1 << 17) + 300
    kp = torch.zeros((n_pages, ps, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros((n_pages, ps, d), dtype=torch.bfloat16, device="cuda")
    c = Case(ns=[1, 3], lens=[700, 300], hq=8, h=2, d=d, ps=ps, dtype="bf16", seed=14)
    far = n_pages - c.c.n_pages
    kp[far:], vp[far:] = c.kp, c.vp
    c.table = torch.where(c.table >= 0, c.table + far, -1).int()
    c.kp, c.vp = kp, vp
    c.c = kvc.cache(n_pages, ps, d, c.table.shape[1], "bf16")
    c.run().check()


def test_tokens_at_far_rows_of_q():
    """A token stride that takes q past 2^31 elements."""
    c = Case(ns=[1, 1], lens=[100, 64], hq=2, h=1, d=64, ps=16, dtype="bf16", seed=15)
    stride = (1 << 31) + 64
    buf = torch.empty(stride + 2 * 64, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((2, 2, 64), (stride, 64, 1))
    q.copy_(c.q)
    c.q = q
    c.run().check()
