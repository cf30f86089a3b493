"""CPU checks of the paged cache's argument validation: everything refused here
is refused on the host before any launch."""
import ctypes as C
import math

import pytest
import torch

NUL, FAKE, ODD = C.c_void_p(0), C.c_void_p(0x1000), C.c_void_p(0x1008)


@pytest.fixture(scope="module")
def kvc():
    from eviction_kvc_score_gb300 import build
    build.build()
    from eviction_kvc_score_gb300 import kvc
    return kvc


GOOD = dict(n_pages=64, page_rows=16, head_dim=64, max_pages=8, dtype="bf16")
BAD = [dict(n_pages=0), dict(n_pages=(1 << 30) + 1), dict(page_rows=8), dict(page_rows=48), dict(head_dim=4),
       dict(head_dim=68), dict(head_dim=264), dict(max_pages=0), dict(max_pages=1 << 27),
       dict(max_pages=(1 << 27) - 15), dict(dtype=7)]


def make(kvc, **kw):
    a = {**GOOD, **kw}
    dt = a.pop("dtype")
    c = kvc.cache(a["n_pages"], a["page_rows"], a["head_dim"], a["max_pages"], "bf16" if dt == 7 else dt)
    if dt == 7:
        c.dtype = 7
    return c


@pytest.mark.parametrize("bad", BAD)
def test_bad_caches_are_refused_everywhere(kvc, bad):
    L, c = kvc._lib, make(kvc, **bad)
    p = C.byref(c)
    assert L.kvc_pages_size(p, 4) == 0
    assert L.kvc_attend_workspace_size(p, 8, 2, 1, 1) == 0
    st = 1 << 40
    assert L.kvc_pages_init(p, FAKE, st, NUL) == -1
    assert L.kvc_pages_status(p, FAKE, st, None, None, NUL) == -1
    assert L.kvc_pages_append(p, FAKE, FAKE, 4, FAKE, FAKE, 1, FAKE, FAKE, 9, FAKE, FAKE, FAKE, st, NUL) == -1
    assert L.kvc_pages_fork(p, FAKE, FAKE, 4, FAKE, FAKE, st, NUL) == -1
    assert L.kvc_pages_compact(p, FAKE, FAKE, 4, FAKE, 3, FAKE, FAKE, FAKE, FAKE, st, NUL) == -1
    assert L.kvc_pages_truncate(p, FAKE, FAKE, 4, FAKE, FAKE, st, NUL) == -1
    assert L.kvc_attend(p, 8, 2, 1, 1, 1, FAKE, 512, FAKE, FAKE, FAKE, FAKE, FAKE, 1.0, FAKE, NUL, FAKE, st, NUL) == -1
    assert kvc.kvc_last_error()


def test_pages_arguments(kvc):
    L, c = kvc._lib, make(kvc)
    p, st = C.byref(c), kvc.kvc_pages_size(make(kvc), 4)
    assert st % 256 == 0 and kvc.kvc_pages_size(c, 400) > st
    assert L.kvc_pages_size(p, 0) == 0 and L.kvc_pages_size(p, (1 << 20) + 1) == 0

    def append(table=FAKE, n=4, k=FAKE, v=FAKE, step=1, rows=9, pool=FAKE, state=FAKE, size=st):
        return L.kvc_pages_append(p, table, FAKE, n, FAKE, FAKE, step, k, v, rows, pool, FAKE, state, size, NUL)
    assert append(table=NUL) == -1 and append(n=0) == -1 and append(k=ODD) == -1 and append(v=NUL) == -1
    assert append(step=-1) == -1 and append(rows=-1) == -1 and append(pool=ODD) == -1
    assert append(state=NUL) == -5 and append(state=C.c_void_p(0x1010)) == -5 and append(size=st - 1) == -5
    assert append(n=400) == -5                                  # a state for 4 lists
    assert L.kvc_pages_fork(p, FAKE, FAKE, 4, NUL, FAKE, st, NUL) == -1
    assert L.kvc_pages_fork(p, FAKE, FAKE, 4, FAKE, FAKE, 256, NUL) == -5
    assert L.kvc_pages_compact(p, FAKE, FAKE, 4, FAKE, 0, FAKE, FAKE, FAKE, FAKE, st, NUL) == -1
    assert L.kvc_pages_compact(p, FAKE, FAKE, 4, FAKE, 3, FAKE, ODD, FAKE, FAKE, st, NUL) == -1
    assert L.kvc_pages_truncate(p, FAKE, NUL, 4, FAKE, FAKE, st, NUL) == -1
    assert L.kvc_pages_init(p, FAKE, 64, NUL) == -5
    assert "kvc_pages_init" in kvc.kvc_last_error()


def test_rope_arguments(kvc):
    L = kvc._lib
    for bad in (dict(rot=0), dict(rot=3), dict(rot=258), dict(theta=0.5), dict(theta=math.inf), dict(theta=math.nan),
                dict(factor=0.5), dict(factor=math.inf), dict(alpha=-1.0), dict(alpha=5.0, beta=4.0), dict(context=0.0),
                dict(alpha=math.nan), dict(beta=math.nan), dict(table=NUL), dict(table=C.c_void_p(0x1004))):
        a = {**dict(rot=64, theta=1e4, factor=2.0, alpha=1.0, beta=4.0, context=100.0, table=FAKE), **bad}
        assert L.kvc_rope_table(a["rot"], a["theta"], a["factor"], a["alpha"], a["beta"], a["context"], a["table"], NUL) == -1, bad

    def rope(dt=1, n=4, hq=2, hk=1, d=64, rot=64, flags=0, pos=FAKE, tab=FAKE, q=FAKE, qs=128, qo=FAKE, qos=128, k=FAKE, ks=64, ko=FAKE, kos=64):
        return L.kvc_rope(dt, n, hq, hk, d, rot, flags, 1.0, pos, tab, q, qs, qo, qos, k, ks, ko, kos, NUL)
    assert rope(n=0) == 0
    for bad in (dict(dt=2), dict(n=-1), dict(n=1 << 31), dict(hq=0, hk=0), dict(hq=-1), dict(d=1, rot=2), dict(rot=66),
                dict(rot=3), dict(rot=0), dict(d=258), dict(flags=4), dict(pos=NUL), dict(tab=NUL), dict(q=NUL), dict(ko=NUL),
                dict(qs=127), dict(kos=63), dict(qos=136), dict(q=C.c_void_p(0x1001)), dict(dt=0, k=C.c_void_p(0x1002))):
        assert rope(**bad) == -1, bad


def test_attend_arguments(kvc):
    L, c = kvc._lib, make(kvc)
    p = C.byref(c)

    def attend(hq=8, h=2, b=1, m=1, n=4, q=FAKE, qs=512, start=FAKE, k=FAKE, scale=0.1, out=FAKE, ws=FAKE, size=1 << 40):
        return L.kvc_attend(p, hq, h, b, m, n, q, qs, start, FAKE, FAKE, k, FAKE, scale, out, NUL, ws, size, NUL)
    for bad in (dict(hq=7), dict(h=0), dict(hq=0), dict(b=0), dict(b=1 << 20), dict(m=0), dict(m=1 << 29), dict(n=-1), dict(n=1 << 31),
                dict(q=NUL), dict(q=ODD), dict(qs=504), dict(qs=513), dict(start=NUL), dict(k=ODD), dict(out=NUL),
                dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38)):
        assert attend(**bad) == -1, bad
    assert L.kvc_attend_workspace_size(p, 8, 3, 1, 1) == 0
    assert L.kvc_attend_workspace_size(p, 8, 2, 0, 1) == 0


def test_without_a_device_calls_end_with_an_error(kvc):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    L, c = kvc._lib, make(kvc, max_pages=(1 << 27) - 16)
    p, st = C.byref(c), 1 << 40
    assert L.kvc_rope_table(64, 1e4, 1.0, 1.0, 4.0, 100.0, FAKE, NUL) == -3
    assert L.kvc_rope(1, 4, 2, 1, 64, 64, 0, 1.0, FAKE, FAKE, FAKE, 128, FAKE, 128, FAKE, 64, FAKE, 64, NUL) == -3
    assert L.kvc_pages_init(p, FAKE, st, NUL) == -3
    assert L.kvc_pages_status(p, FAKE, st, None, None, NUL) == -3
    assert L.kvc_pages_append(p, FAKE, FAKE, 4, FAKE, FAKE, 1, FAKE, FAKE, 9, FAKE, FAKE, FAKE, st, NUL) == -3
    assert L.kvc_pages_fork(p, FAKE, FAKE, 4, FAKE, FAKE, st, NUL) == -3
    assert L.kvc_pages_compact(p, FAKE, FAKE, 4, FAKE, 3, FAKE, FAKE, FAKE, FAKE, st, NUL) == -3
    assert L.kvc_pages_truncate(p, FAKE, FAKE, 4, FAKE, FAKE, st, NUL) == -3
    assert L.kvc_attend(p, 8, 2, 1, 1, 1, FAKE, 512, FAKE, FAKE, FAKE, FAKE, FAKE, 1.0, FAKE, NUL, FAKE, st, NUL) == -3
    assert "kvc_attend" in kvc.kvc_last_error()


def test_binding_refuses_wrong_tensors(kvc):
    """Host tensors, wrong types and shapes never reach the library."""
    c = make(kvc)
    host = torch.zeros((4, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        kvc.kvc_pages_truncate(c, host, torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), host)
    with pytest.raises(ValueError):
        kvc.kvc_pages_truncate(c, torch.zeros((4, 9), dtype=torch.int32), host, host, host)
    x = torch.zeros((3, 2, 64))
    with pytest.raises(ValueError):
        kvc.kvc_rope(torch.zeros(32, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), x, None, x, None, 64)
    with pytest.raises(ValueError):
        kvc.kvc_rope(torch.zeros(32, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), None, None, None, None, 64)
    with pytest.raises(ValueError):
        kvc.kvc_rope(torch.zeros(32, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), x.half(), None, x.half(), None, 64)
    with pytest.raises(ValueError):
        kvc.kvc_rope(torch.zeros(32, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), x, None, None, None, 64)
    with pytest.raises(ValueError):
        kvc.cache(4, 16, 64, 4, torch.float16)
