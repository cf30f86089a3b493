"""Few lists that move rows among very many that do not."""
import pytest
import torch

from test_pages_gpu import Real, K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def rows_of(real, i, n):
    pages = real.table[i, :-(-n // real.c.page_rows)].long()
    return real.kp[pages].reshape(-1, real.c.head_dim)[:n, 0], real.vp[pages].reshape(-1, real.c.head_dim)[:n, 0]


def test_rows_between_hundreds_of_thousands_of_empty_lists():
    """Two long lists and a short one far apart: every warp whose run of rows or of pages passes from
    one to the next finds it at once.  (One list after the other, that was 160,000 loads in a row and 15 ms a
    call; it takes 0.43 ms, most of it the plan's pass over the lists.)"""
    lists, n = 1 << 18, 12000
    at = [5, 100000, lists - 3]
    counts = [n, 3, n]
    real = Real(600, 128, 94, lists, dim=8)
    src = torch.arange(1, sum(counts) + 1, device="cuda", dtype=torch.float32)[:, None].expand(-1, 8).contiguous()
    count = torch.zeros(lists, dtype=torch.int32, device="cuda")
    first = torch.zeros(lists, dtype=torch.int64, device="cuda")
    count[at] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    first[at] = torch.tensor([0, n, n + 3], device="cuda")
    none = torch.zeros(lists, dtype=torch.int32, device="cuda")

    def append():
        K().kvc_pages_append(real.c, real.table, real.len, count, first, 1, src, -src, real.kp, real.vp, real.state)

    def check(ns):
        begin = 0
        for i, c, m in zip(at, counts, ns):
            k, v = rows_of(real, i, m)
            assert torch.equal(k, src[begin:begin + m, 0]) and torch.equal(v, -k), i
            begin += c
        assert real.status() == (0, 600 - sum(-(-m // 128) for m in ns))
        assert int(real.len.sum()) == sum(ns)

    def timed(f):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b)
    times = []
    for again in range(3):
        K().kvc_pages_truncate(real.c, real.table, real.len, none, real.state)
        times.append(timed(append))
        check(counts)
    # and one row of each kept
    idx = torch.zeros((lists, 1), dtype=torch.int32, device="cuda")
    one = torch.full((lists,), -1, dtype=torch.int32, device="cuda")
    one[at] = 1
    K().kvc_pages_compact(real.c, real.table, real.len, idx, one, real.kp, real.vp, real.state)
    check([1, 1, 1])
    assert min(times) < 5.0, times
