"""Rows held in 4 or 8 bits, written, moved and read back: what is read is what
the format's definition says, value for value."""
import math

import pytest
import torch

import cache_ref
import quant_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def i64(x):
    return torch.tensor(x, dtype=torch.int64, device="cuda")


class Cache:
    def __init__(self, n_pages, ps, max_pages, n_lists, d, dtype, bits, seed=0):
        kvc = K()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bits, self.dt = bits, DT[dtype]
        self.c = kvc.cache(n_pages, ps, d, max_pages, dtype)
        self.state = torch.empty(kvc.kvc_pages_size(self.c, n_lists), dtype=torch.uint8, device="cuda")
        kvc.kvc_pages_init(self.c, self.state)
        size = kvc.kvc_quant_page_size(self.c, bits)
        # whatever the pools hold before: random bytes
        self.kp, self.vp = (torch.randint(0, 256, (n_pages, size), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
        self.table = torch.full((n_lists, max_pages), -1, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(n_lists, dtype=torch.int32, device="cuda")

    def append(self, counts, row, step, k, v, **kw):
        K().kvc_pages_append_quant(self.c, self.bits, self.table, self.len, i32(counts), i64(row), step, k, v, self.kp, self.vp, self.state, **kw)

    def compact(self, idx, counts):
        K().kvc_pages_compact_quant(self.c, self.bits, self.table, self.len, i32(idx), i32(counts), self.kp, self.vp, self.state)

    def read(self, first, counts, row, step, rows, fill=7.0, want=(True, True), table=None, state=None):
        d = self.c.head_dim
        out = [torch.full((rows, d), fill, dtype=self.dt, device="cuda") if w else None for w in want]
        K().kvc_pages_read_quant(self.c, self.bits, self.table if table is None else table, self.len,
                                 None if first is None else i32(first), i32(counts), i64(row), step,
                                 self.kp if want[0] else None, self.vp if want[1] else None, *out, self.state if state is None else state)
        return out

    def lists(self):
        """Every list's K and V, read one after the other."""
        n = self.len.tolist()
        at = [sum(n[:i]) for i in range(len(n))]
        k, v = self.read(None, n, [a if x else 0 for a, x in zip(at, n)], 1, max(1, sum(n)))
        return [(k[a:a + x], v[a:a + x]) for a, x in zip(at, n)]

    def status(self):
        return K().kvc_pages_status(self.c, self.state)


def same(a, b):
    """Equal, and NaN in the same places."""
    a, b = a.double(), b.double()
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def rows_of(g, n, d, dt):
    """Random rows of many sizes, some channels strong and off zero, some rows one-sided, some groups zero."""
    x = torch.randn((n, d), generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (n, 1), generator=g, device="cuda").float())
    x[:, ::37] = 5 * x[:, ::37] + 3
    x[::5] = x[::5].abs()
    x[1::7, :32] = 0
    x[2::7, -8:] = -x[2::7, -8:].abs()
    return x.to(dt)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,ps", [(8, 16), (32, 128), (40, 32), (64, 16), (80, 64), (128, 16), (128, 64), (200, 32), (256, 128)])
def test_rows_read_back_as_defined(d, ps, dtype, bits):
    lens, n_lists = [0, 1, 15, 16, 17, 3 * ps + 5, 260, 2, 0, ps], 10
    x = Cache(80, ps, 300 // ps + 2, n_lists, d, dtype, bits, seed=d)
    g = torch.Generator(device="cuda").manual_seed(d + bits)
    held = [(torch.zeros((0, d), dtype=x.dt, device="cuda"),) * 2 for _ in range(n_lists)]
    for part in range(3):    # three appends, token-major rows with others between
        step = part + 1
        counts = [(n + 2 - part) // 3 for n in lens]
        starts = [2 + sum(counts[:i]) * step for i in range(n_lists)]
        src = [rows_of(g, 2 + sum(counts) * step, d, x.dt) for _ in range(2)]
        x.append(counts, starts, step, *src)
        for i, (s, n) in enumerate(zip(starts, counts)):
            if n:
                held[i] = tuple(torch.cat([h, y[s:s + (n - 1) * step + 1:step]]) for h, y in zip(held[i], src))
    assert x.len.tolist() == lens
    want = [tuple(ref.stands(y, bits) for y in h) for h in held]
    for got, w in zip(x.lists(), want):
        assert same(got[0], w[0]) and same(got[1], w[1])
    # a stretch of each list, to rows two apart; the rows between stay as they are
    first = [n // 3 for n in lens]
    counts = [n - n // 3 - n // 5 for n in lens]
    at = [1 + 2 * sum(counts[:i]) for i in range(n_lists)]
    for only in ((True, True), (True, False), (False, True)):
        out = x.read(first, counts, at, 2, 2 * sum(counts) + 1, want=only)
        for j, o in enumerate(out):
            if o is None:
                continue
            assert (o[0::2] == 7).all()
            for i, n in enumerate(counts):
                assert same(o[at[i]:at[i] + 2 * n:2], want[i][j][first[i]:first[i] + n])
    assert x.status()[0] == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_groups_where_the_format_ends(dtype, bits):
    """Zeros of either sign, one value, one side, subnormal and huge values, ties,
    infinities and NaN: a group each, the neighbours untouched by them."""
    big, n = 2.0 ** 126, ref.N[bits]
    top = torch.finfo(DT[dtype]).max
    groups = [[0.0] * 32, [-0.0] * 32, [3.0] * 32, [-3.0] * 32, [1.0] + [0.0] * 31, [-1.0] + [0.0] * 31,
              [float(i) for i in range(32)], [float(i - 31) for i in range(32)], [i / 2 for i in range(-16, 16)],
              [1e-40] * 16 + [-1e-39] * 16, [2.0 ** -126] * 32, [2.0 ** -149] * 32, [2.0 ** -120, -2.0 ** -121] * 16,
              [big * 0.99] * 16 + [-big * 0.99] * 16, [big] + [1.0] * 31, [1.0] * 31 + [-big], [top] * 32,
              [math.inf] + [0.0] * 31, [0.0] * 31 + [-math.inf], [math.nan] * 32, [1.0] * 16 + [math.nan] + [1.0] * 15,
              [math.nan, math.inf] * 16, [n * 1.0] + [i + 0.5 for i in range(15)] + [0.0] * 16,
              [n + 0.001] + [-1.5] * 31, [1e30] + [1e-30] * 31]
    d = 256
    flat = sum((x if i % 2 else x[::-1] for i, x in enumerate(groups)), [])
    flat += [1.0] * (-len(flat) % d)
    y = torch.tensor(flat, device="cuda").to(DT[dtype]).view(-1, d)
    # every group once in every place of a row
    rows = torch.cat([y.view(-1, 8, 32).roll(i, 1).reshape(-1, d) for i in range(8)])
    x = Cache(8, 32, 8, 1, d, dtype, bits)
    x.append([rows.shape[0]], [0], 1, rows, rows.flip(0).contiguous())
    (k, v), = x.lists()
    want = ref.stands(rows, bits)
    assert same(k, want) and same(v, want.flip(0))
    fine = want.isfinite()
    step = ref.quantise(rows, bits)[1]
    assert ((want - rows.double()).abs() <= step * 1.001)[fine].all()   # one step where the code is cut, half elsewhere
    assert (k.double()[(rows == 0) & fine] == 0).all()


@pytest.mark.parametrize("bits,d,dtype", [(4, 128, "bf16"), (8, 80, "f32"), (4, 40, "f32")])
def test_sharing_evicting_and_giving_back(bits, d, dtype):
    """Fork, copy on write, compaction and truncation with the rows' values, against
    a list model of the pool (pages as well as values)."""
    ps, n_pages, n_lists = 16, 64, 6
    x, model = Cache(n_pages, ps, 16, n_lists, d, dtype, bits), cache_ref.Pages(n_pages, ps, 16, n_lists)
    g = torch.Generator(device="cuda").manual_seed(5)
    src = [rows_of(g, 400, d, x.dt) for _ in range(2)]
    want = [ref.stands(y, bits) for y in src]
    used = 0

    def append(counts):
        nonlocal used
        at = [used + sum(counts[:i]) for i in range(n_lists)]
        used += sum(counts)
        assert model.append([list(range(a, a + n)) for a, n in zip(at, counts)])
        x.append(counts, at, 1, *src)

    def check():
        for i, got in enumerate(x.lists()):
            rows = i64(model.list_rows(i))
            assert x.table[i, :len(model.table[i])].tolist() == model.table[i]
            assert same(got[0], want[0][rows]) and same(got[1], want[1][rows])
        assert x.status() == (0, len(model.free()))

    append([37, 0, 20, 0, 0, 1])
    check()
    fork = [-1, 0, -1, 0, 2, -1]
    model.fork(fork)
    K().kvc_pages_fork(x.c, x.table, x.len, i32(fork), x.state)
    check()
    append([1, 2, 0, 17, 13, 15])
    check()
    idx = [None, [38, 0, 7, 7], None, list(range(53, 0, -3)), [], list(range(16))]
    assert model.compact(idx)
    m = max(len(r) for r in idx if r)
    x.compact([(r or []) + [-5] * (m - len(r or [])) for r in idx], [-1 if r is None else len(r) for r in idx])
    check()
    append([20, 1, 3, 0, 30, 1])
    check()
    new = [5, -1, 0, 16, 7, 40]
    model.truncate(new)
    K().kvc_pages_truncate(x.c, x.table, x.len, i32(new), x.state)
    check()
    append([3, 3, 3, 3, 3, 3])
    check()


def test_calls_that_do_not_fit_change_nothing():
    kvc = K()
    x = Cache(4, 16, 3, 3, 64, "bf16", 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    src = [rows_of(g, 100, 64, x.dt) for _ in range(2)]
    x.append([20, 5, 0], [0, 20, 0], 1, *src)
    before = [t.clone() for t in (x.kp, x.vp, x.table, x.len)]

    def unchanged(bits):
        assert x.status()[0] & bits == bits
        assert all(torch.equal(a, b) for a, b in zip(before, (x.kp, x.vp, x.table, x.len)))
        free = x.status()[1]
        assert free == 1

    x.append([13, 12, 1], [0, 0, 0], 1, *src)              # three pages wanted, one is free
    unchanged(kvc.DEV_PAGES_FULL)
    x.append([1, 1, 0], [0, 100, 0], 1, *src)              # a source row behind the last
    unchanged(kvc.DEV_BAD_LIST)
    x.append([3, 0, 0], [0, 0, 0], 50, *src)
    unchanged(kvc.DEV_BAD_LIST)
    x.append([29, 0, 0], [0, 0, 0], 1, *src)               # more than max_pages hold
    unchanged(kvc.DEV_PAGES_FULL)
    x.compact([[0] * 40, [0] * 40, [0] * 40], [17, 17, -1])   # four pages wanted
    unchanged(kvc.DEV_PAGES_FULL)
    for first, counts, row, step, rows in (([0, 1, 0], [20, 5, 0], [0, 20, 0], 1, 30), ([-1, 0, 0], [2, 0, 0], [0, 0, 0], 1, 30),
                                           ([0, 0, 0], [2, 0, 0], [29, 0, 0], 1, 30), ([0, 0, 0], [3, 0, 0], [0, 0, 0], 15, 30),
                                           ([0, 0, 0], [1, 0, 0], [-1, 0, 0], 1, 30), ([0, 0, 0], [0, 0, 1], [0, 0, 0], 1, 30),
                                           ([2 ** 31 - 1, 0, 0], [2 ** 31 - 1, 0, 0], [0, 0, 0], 1, 30)):
        state = torch.empty_like(x.state)     # a state of its own: its status is this call's
        kvc.kvc_pages_init(x.c, state)
        for o in x.read(first, counts, row, step, rows, state=state):
            assert (o == 7).all()
        assert kvc.kvc_pages_status(x.c, state)[0] == kvc.DEV_BAD_LIST


def test_what_tables_and_indexes_get_wrong():
    """Pages outside the pool are rows of zeros when read; an index outside a list
    gives a row of zeros when compacted."""
    kvc = K()
    x = Cache(16, 16, 4, 2, 96, "bf16", 8)
    g = torch.Generator(device="cuda").manual_seed(2)
    src = [rows_of(g, 80, 96, x.dt) for _ in range(2)]
    x.append([40, 40], [0, 40], 1, *src)
    want = [ref.stands(y, 8) for y in src]
    table = x.table.clone()
    table[0, 1], table[1, 2] = 16, -3
    k, v = x.read(None, [40, 40], [0, 40], 1, 80, table=table)
    for got, w in ((k, want[0]), (v, want[1])):
        w = w.clone()
        w[16:32], w[72:80] = 0, 0
        assert same(got, w)
    assert x.status()[0] == kvc.DEV_BAD_PAGE
    x.compact([[3, 40, -1, 39], [0, 1, 2, 3]], [4, -1])
    assert x.status()[0] == kvc.DEV_BAD_PAGE | kvc.DEV_BAD_LIST
    k, v = x.lists()[0]
    for got, w in ((k, want[0]), (v, want[1])):
        assert same(got, torch.stack([w[3], 0 * w[0], 0 * w[0], w[39]]))


def test_many_lists_most_of_them_empty():
    """More lists than the plan's block has threads, a few of them with rows."""
    n_lists, d = 5000, 64
    x = Cache(200, 16, 40, n_lists, d, "bf16", 4)
    g = torch.Generator(device="cuda").manual_seed(3)
    some = {0: 3, 17: 600, 1023: 1, 1024: 40, 4998: 500}
    counts = [some.get(i, 0) for i in range(n_lists)]
    at = {i: sum(n for j, n in some.items() if j < i) for i in some}
    src = [rows_of(g, sum(counts), d, x.dt) for _ in range(2)]
    x.append(counts, [at.get(i, 0) for i in range(n_lists)], 1, *src)
    k, v = x.read(None, counts, [at.get(i, 0) for i in range(n_lists)], 1, sum(counts))
    assert same(k, ref.stands(src[0], 4)) and same(v, ref.stands(src[1], 4))


def test_no_rows_at_all():
    x = Cache(4, 16, 2, 2, 64, "f32", 4)
    empty = torch.zeros((0, 64), device="cuda")
    x.append([0, -3], [0, 0], 1, empty, empty)
    k, v = x.read(None, [0, 0], [0, 0], 1, 0)
    assert k.shape[0] == 0 and x.len.tolist() == [0, 0] and x.status() == (0, 4)


def test_captured_and_replayed_on_another_stream():
    kvc = K()
    d, lists = 128, 4
    x = Cache(60, 16, 16, lists, d, "bf16", 4)
    g = torch.Generator(device="cuda").manual_seed(4)
    src = [rows_of(g, 64, d, x.dt) for _ in range(2)]
    counts, row, first = i32([3, 0, 1, 16]), i64([0, 0, 5, 9]), i32([0] * lists)
    to = i64([0, 0, 8, 16])
    out = [torch.zeros((40, d), dtype=x.dt, device="cuda") for _ in range(2)]

    def step():
        kvc.kvc_pages_append_quant(x.c, 4, x.table, x.len, counts, row, 1, *src, x.kp, x.vp, x.state)
        kvc.kvc_pages_read_quant(x.c, 4, x.table, x.len, first, counts, to, 1, x.kp, x.vp, *out, x.state)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        side.synchronize()
        for n in range(2, 4):
            for y in src:
                y.mul_(-1.25)
            graph.replay()
            side.synchronize()
            assert x.len.tolist() == [3 * n, 0, n, 16 * n]
        # the rows at the lists' beginnings are the first call's
        first.copy_(x.len - counts)
        kvc.kvc_pages_read_quant(x.c, 4, x.table, x.len, first, counts, to, 1, x.kp, x.vp, *out, x.state)
    side.synchronize()
    for o, y in zip(out, src):
        w = ref.stands(y, 4)
        assert same(o[0:3], w[0:3]) and same(o[8:9], w[5:6]) and same(o[16:32], w[9:25])
    assert x.status()[0] == 0


def test_the_last_page_of_a_large_pool():
    """Bytes behind 2^32 of a pool (a table made by hand: what the allocator would
    only get to after every page before)."""
    d, ps = 256, 128
    kvc = K()
    n_pages = 2 ** 32 // (128 * 272) + 3
    x = Cache.__new__(Cache)
    x.bits, x.dt = 8, torch.bfloat16
    x.c = kvc.cache(n_pages, ps, d, 4, "bf16")
    x.state = torch.empty(kvc.kvc_pages_size(x.c, 1), dtype=torch.uint8, device="cuda")
    kvc.kvc_pages_init(x.c, x.state)
    size = kvc.kvc_quant_page_size(x.c, 8)
    assert n_pages * size > 2 ** 32
    x.kp, x.vp = (torch.empty((n_pages, size), dtype=torch.uint8, device="cuda") for _ in range(2))
    x.table, x.len = torch.full((1, 4), -1, dtype=torch.int32, device="cuda"), i32([0])
    g = torch.Generator(device="cuda").manual_seed(6)
    src = [rows_of(g, 130, d, x.dt) for _ in range(2)]
    x.append([130], [0], 1, *src)
    for p in (x.kp, x.vp):
        p[n_pages - 1].copy_(p[0])
        p[0].zero_()
    x.table[0, 0] = n_pages - 1
    k, v = x.read(None, [130], [0], 1, 130)
    assert same(k, ref.stands(src[0], 8)) and same(v, ref.stands(src[1], 8))
    # and written there: 100 rows cut off and put back
    kvc.kvc_pages_truncate(x.c, x.table, x.len, i32([30]), x.state)
    x.append([98], [30], 1, *src)
    k, v = x.read(None, [128], [0], 1, 128)
    assert same(k, ref.stands(src[0][:128], 8)) and same(v, ref.stands(src[1][:128], 8))
