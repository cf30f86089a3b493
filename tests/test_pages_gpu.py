"""Page moves against a plain model of the pool: tables, lengths, row bytes and
free pages after every call are equal, not close."""
import random

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


class Real:
    """The library's side: rows are numbers r, held as r in every element of K and -r of V."""

    def __init__(self, n_pages, ps, max_pages, n_lists, dim=64, dtype="f32"):
        kvc = K()
        self.c = kvc.cache(n_pages, ps, dim, max_pages, dtype)
        self.state = torch.empty(kvc.kvc_pages_size(self.c, n_lists), dtype=torch.uint8, device="cuda")
        kvc.kvc_pages_init(self.c, self.state)
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.kp = torch.zeros((n_pages, ps, dim), dtype=dt, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.table = torch.full((n_lists, max_pages), -1, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(n_lists, dtype=torch.int32, device="cuda")

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def append(self, rows, step=1):
        flat, start = [0.0], []
        for new in rows:     # step > 1: other rows lie between
            start.append(len(flat))
            for r in new:
                flat += [float(r)] + [9e5] * (step - 1)
        src = torch.tensor(flat, device="cuda")[:, None].expand(-1, self.c.head_dim).contiguous().to(self.kp.dtype)
        start = [s if rows[i] else 0 for i, s in enumerate(start)]
        K().kvc_pages_append(self.c, self.table, self.len, self.i32([len(x) for x in rows]),
                             torch.tensor(start, dtype=torch.int64, device="cuda"), step, src, -src, self.kp, self.vp, self.state)

    def fork(self, src):
        K().kvc_pages_fork(self.c, self.table, self.len, self.i32(src), self.state)

    def compact(self, idx):
        m = max([1] + [len(x) for x in idx if x is not None])
        k = [[-7] * m if x is None else list(x) + [-7] * (m - len(x)) for x in idx]
        K().kvc_pages_compact(self.c, self.table, self.len, self.i32(k), self.i32([-1 if x is None else len(x) for x in idx]),
                              self.kp, self.vp, self.state)

    def truncate(self, new):
        K().kvc_pages_truncate(self.c, self.table, self.len, self.i32(new), self.state)

    def status(self):
        return K().kvc_pages_status(self.c, self.state)


def same(real, model, status=0):
    assert real.status() == (status, len(model.free()))
    assert real.len.tolist() == model.len
    table, kp, vp = real.table.cpu(), real.kp.cpu(), real.vp.cpu()
    for i, pages in enumerate(model.table):
        assert table[i, :len(pages)].tolist() == pages, i
        if not model.len[i]:
            continue
        want = torch.tensor(model.list_rows(i), dtype=torch.float32)[:, None]
        for pool, sign in ((kp, 1), (vp, -1)):
            got = pool[torch.tensor(pages)].reshape(-1, real.c.head_dim)[:model.len[i]].float()
            assert torch.equal(got, (sign * want).expand_as(got)), i


def pair(*a, **k):
    m = ref.Pages(*a)
    return Real(*a, **k), m


@pytest.mark.parametrize("seed,ps,dim,dtype", [(0, 16, 64, "f32"), (1, 16, 8, "bf16"), (2, 32, 80, "bf16"), (3, 64, 256, "f32"),
                                              (4, 128, 128, "bf16"), (5, 16, 40, "f32"), (6, 64, 24, "bf16")])
def test_random_histories(seed, ps, dim, dtype):
    """Appends, forks, cuts and compactions in any order, some too large for the pool."""
    rnd = random.Random(seed)
    lists = 13
    real, model = pair(60, ps, 9, lists, dim=dim, dtype=dtype)
    row, full = 1, 0
    for step in range(60):
        kind = rnd.choice(["append", "append", "fork", "compact", "truncate"])
        if kind == "append":
            rows = []
            for i in range(lists):
                n = rnd.choice([0, 0, 1, 2, ps, rnd.randint(1, 3 * ps)])
                rows.append([(row + j) % 250 + 1 for j in range(n)])   # exact in bf16
                row += n
            real.append(rows, step=rnd.choice([1, 3]))
            if not model.append(rows):
                full = 0x80
        elif kind == "fork":
            src = [-1] * lists
            empty = [i for i in range(lists) if model.len[i] == 0]
            for i in rnd.sample(empty, min(len(empty), 4)):
                src[i] = rnd.choice([j for j in range(lists) if j not in empty] or [-1])
            real.fork(src)
            model.fork(src)
        elif kind == "compact":
            idx = []
            for i in range(lists):
                n = model.len[i]
                keep = rnd.choice([None, None, rnd.randint(0, n)])
                idx.append(None if keep is None else sorted(rnd.sample(range(n), keep)) if rnd.random() < 0.7 else
                           [rnd.randrange(n) for _ in range(keep)])
            real.compact(idx)
            if not model.compact(idx):
                full = 0x80
        else:
            new = [rnd.choice([-1, -1, 0, rnd.randint(0, max(1, model.len[i])), 1 << 20]) for i in range(lists)]
            real.truncate(new)
            model.truncate(new)
        same(real, model, full)
    real.truncate([0] * lists)
    model.truncate([0] * lists)
    same(real, model, full)
    assert real.status()[1] == 60


def test_shared_last_pages_are_copied_by_each_appender():
    real, model = pair(40, 16, 6, 5)
    for step in (lambda x: x.append([list(range(1, 22)), [], [], [], []]),
                 lambda x: x.fork([-1, 0, 0, -1, -1]),
                 lambda x: x.append([[101], [102], [], [], []]),      # both write behind the shared page
                 lambda x: x.append([[], [103], [104], [], []]),      # the third is its page's last holder
                 lambda x: x.truncate([17, -1, 3, -1, -1]),
                 lambda x: x.fork([-1, -1, -1, 1, 0]),
                 lambda x: x.append([[105] * 40, [106] * 16, [107], [108], [109]])):
        step(real)
        step(model)
        same(real, model)


def test_all_or_nothing():
    real, model = pair(6, 16, 4, 3)
    real.append([[1] * 30, [2] * 16, []])
    model.append([[1] * 30, [2] * 16, []])
    before = real.table.clone(), real.kp.clone(), real.len.clone()
    for rows in ([[3], [4], [5] * 49], [[1] * 35, [], []]):   # six pages hold no more; four entries do not
        real.append(rows)
        assert real.status() == (0x80, 3)
        for a, b in zip(before, (real.table, real.kp, real.len)):
            assert torch.equal(a, b)
    real.compact([list(range(30)), list(range(16)), []])      # three fresh pages: just fits
    model.compact([list(range(30)), list(range(16)), []])
    same(real, model, 0x80)


def test_bad_arguments_on_the_device_change_nothing():
    kvc = K()
    for what in ("len", "neg_len", "src", "src_far", "page", "k_max"):
        real, model = pair(12, 16, 4, 2)
        real.append([[1] * 20, [2] * 5])
        src = torch.ones((10, 64), device="cuda")
        counts, rows = real.i32([1, 3]), torch.tensor([0, 7], dtype=torch.int64, device="cuda")
        status = 0x20
        if what == "len":
            real.len[1] = 65
        elif what == "neg_len":
            real.len[0] = -1
        elif what == "src":
            rows[0] = -1
        elif what == "src_far":
            rows[1] = 8
        elif what == "page":
            real.table[0, 1], status = 12, 0x40
        before = real.table.clone(), real.kp.clone(), real.len.clone()
        if what == "k_max":
            idx = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
            kvc.kvc_pages_compact(real.c, real.table, real.len, idx, counts, real.kp, real.vp, real.state)
        else:
            kvc.kvc_pages_append(real.c, real.table, real.len, counts, rows, 1, src, src, real.kp, real.vp, real.state)
        assert real.status() == (status, 9), what
        for a, b in zip(before, (real.table, real.kp, real.len)):
            assert torch.equal(a, b), what


def test_bad_entries_are_skipped():
    real, _ = pair(12, 16, 4, 4)
    real.append([[1] * 20, [], [], []])
    real.fork([-1, 0, 1, 9])            # list 1 from 0; 2 from a list forked into; 3 from none
    assert real.status()[0] == 0x20 and real.len.tolist() == [20, 20, 0, 0]
    K().kvc_pages_init(real.c, real.state)
    real.len.zero_()
    real.append([[1] * 20, [2], [], []])
    real.fork([1, -1, -1, -1])          # not empty
    assert real.status()[0] == 0x20 and real.len.tolist() == [20, 1, 0, 0]
    # rows outside the list come as zeros
    K().kvc_pages_init(real.c, real.state)
    real.len.zero_()
    real.append([[3] * 20, [], [], []])
    real.compact([[19, -1, 20, 0], None, None, None])
    assert real.status()[0] == 0x20
    got = real.kp[real.table[0, 0].item(), :4, 0].tolist()
    assert got == [3, 0, 0, 3]
    # a page let go of twice is counted once
    K().kvc_pages_init(real.c, real.state)
    real.len.zero_()
    real.append([[1] * 16, [], [], []])
    real.table[1] = real.table[0]
    real.len[1] = 16
    real.truncate([0, -1, -1, -1])
    real.truncate([-1, 0, -1, -1])
    assert real.status() == (0x40, 12)
    # entries outside the pool are passed over
    K().kvc_pages_init(real.c, real.state)
    real.table[2, 0], real.table[2, 1] = -5, 99
    real.len.copy_(real.i32([0, 0, 32, 0]))
    real.truncate([-1, -1, 0, -1])
    assert real.status() == (0x40, 12)


def test_many_lists_and_a_pool_of_several_groups():
    """Thousands of lists; free pages scattered over a pool of 100,000."""
    lists, ps = 5000, 16
    real = Real(100000, ps, 16, lists, dim=8)
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 200, (lists,), generator=g)
    src = torch.arange(int(counts.sum()) + 1, device="cuda", dtype=torch.float32)[:, None].expand(-1, 8).contiguous()
    row = (counts.cumsum(0) - counts).cuda()
    kvc = K()
    kvc.kvc_pages_append(real.c, real.table, real.len, counts.int().cuda(), row, 1, src, -src, real.kp, real.vp, real.state)
    pages = (counts + ps - 1) // ps
    first = pages.cumsum(0) - pages
    taken = int(pages.sum())
    assert real.status() == (0, 100000 - taken)
    at = torch.arange(16)
    want = torch.where(at < pages[:, None], first[:, None] + at, -1)
    assert torch.equal(real.table.cpu().long(), want)
    # every third list freed, then all of it asked for again, and more
    third = torch.arange(lists) % 3 == 0
    kvc.kvc_pages_truncate(real.c, real.table, real.len, torch.where(third, 0, -1).int().cuda(), real.state)
    holes = torch.cat([torch.arange(int(first[i]), int(first[i] + pages[i])) for i in torch.nonzero(third).view(-1)])
    free = torch.cat([holes, torch.arange(taken, 100000)])
    assert real.status()[1] == free.numel()
    again = torch.where(third, 250, 0)
    row = (again.cumsum(0) - again).cuda()
    src = torch.randn((int(again.sum()), 8), device="cuda")
    kvc.kvc_pages_append(real.c, real.table, real.len, again.int().cuda(), row, 1, src, src, real.kp, real.vp, real.state)
    n = int(third.sum()) * 16
    got = real.table.cpu()[third].reshape(-1).long()
    assert torch.equal(got, free[:n])
    rows = real.kp[got.cuda()].reshape(-1, 256, 8)[:, :250].reshape(-1, 8)
    assert torch.equal(rows, src)
    assert real.status() == (0, free.numel() - n)


def test_thousands_of_lists_compacted_and_appended_to_while_shared():
    """Plans of more lists than one block has threads, with copied last pages."""
    kvc, lists, ps = K(), 3000, 16
    real = Real(60000, ps, 8, lists, dim=8)
    g = torch.Generator().manual_seed(6)
    half = lists // 2
    n = torch.randint(1, 100, (half,), generator=g)
    counts = torch.cat([n, torch.zeros(half, dtype=torch.int64)])
    src = torch.randn((int(n.sum()), 8), generator=g).cuda()
    row = (counts.cumsum(0) - counts).cuda()
    kvc.kvc_pages_append(real.c, real.table, real.len, counts.int().cuda(), row, 1, src, src, real.kp, real.vp, real.state)
    fork = torch.cat([torch.full((half,), -1), torch.arange(half)]).int().cuda()
    kvc.kvc_pages_fork(real.c, real.table, real.len, fork, real.state)
    pages = (n + ps - 1) // ps
    used = int(pages.sum())
    assert real.status() == (0, 60000 - used)
    # every list takes one row: both holders of a partly filled page copy it,
    # and its old page is nobody's
    more = torch.randn((lists, 8), generator=g).cuda()
    ones = torch.ones(lists, dtype=torch.int32, device="cuda")
    kvc.kvc_pages_append(real.c, real.table, real.len, ones, torch.arange(lists, device="cuda"), 1, more, more, real.kp, real.vp, real.state)
    part = n % ps > 0
    now = 2 * int(torch.where(part, pages, pages + 1).sum()) - int(torch.where(part, pages - 1, pages).sum())
    assert real.status() == (0, 60000 - now)

    def rows(i):
        at = int(real.len[i])
        return real.kp[real.table[i, :-(-at // ps)].long()].reshape(-1, 8)[:at]
    first = n.cumsum(0) - n
    for i in (0, 1, 777, half - 1, half, half + 777, lists - 1):
        j = i % half
        assert torch.equal(rows(i), torch.cat([src[first[j]:first[j] + n[j]], more[i:i + 1]]))
    # the forks keep every other row, last first
    m = int(n.max()) + 1
    keep = (real.len.cpu()[half:].long() + 1) // 2
    idx = (real.len[half:, None] - 1 - 2 * torch.arange(m, device="cuda")).int()
    idx = torch.cat([torch.zeros((half, m), dtype=torch.int32, device="cuda"), idx]).contiguous()
    counts = torch.cat([torch.full((half,), -1), keep]).int().cuda()
    before = {i: rows(i).clone() for i in (0, 5, half, half + 5, lists - 1)}
    kvc.kvc_pages_compact(real.c, real.table, real.len, idx, counts, real.kp, real.vp, real.state)
    for i, old in before.items():
        assert torch.equal(rows(i), old if i < half else old.flip(0)[::2])
    kvc.kvc_pages_truncate(real.c, real.table, real.len, torch.zeros_like(real.len), real.state)
    assert real.status() == (0, 60000)


def test_more_pages_than_32_bits_count():
    """Requests whose sum passes 2^32 pages are refused, not wrapped."""
    real = Real(64, 16, 1 << 20, 5000, dim=8)
    real.append([[1] * 3] + [[]] * 4999)
    counts = torch.full((5000,), (1 << 24) - 5, dtype=torch.int32, device="cuda")
    src = torch.zeros((1 << 24, 8), device="cuda")
    row = torch.zeros(5000, dtype=torch.int64, device="cuda")
    K().kvc_pages_append(real.c, real.table, real.len, counts, row, 1, src, src, real.kp, real.vp, real.state)
    assert real.status() == (0x80, 63) and real.len.sum().item() == 3


def test_layer_views_streams_and_graphs():
    """One layer's lists out of a larger table, on another stream, captured and replayed."""
    kvc = K()
    real, model = pair(64, 16, 4, 6)
    rows = [[], [], [5], [6], [], []]
    src = torch.tensor([5.0, 6.0], device="cuda")[:, None].expand(-1, 64).contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    count, row = real.i32([1, 1]), torch.tensor([0, 1], dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kvc.kvc_pages_append(real.c, real.table[2:4], real.len[2:4], count, row, 1, src, -src, real.kp, real.vp, real.state)
    for _ in range(40):
        graph.replay()
        model.append(rows)
    torch.cuda.synchronize()
    same(real, model)


def test_state_for_more_lists_serves_fewer():
    """The state's layout does not depend on a call's number of lists."""
    real, model = pair(64, 16, 4, 6)
    real.append([[1] * 20, [2], [], [], [3] * 5, []])
    model.append([[1] * 20, [2], [], [], [3] * 5, []])
    one = torch.tensor([17], dtype=torch.int32, device="cuda")
    K().kvc_pages_truncate(real.c, real.table[:1], real.len[:1], one, real.state)
    model.truncate([17, -1, -1, -1, -1, -1])
    same(real, model)
