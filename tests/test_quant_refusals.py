"""CPU checks of what the calls on a cache held in 4 or 8 bits refuse: nothing is
launched, and the message names the call."""
import ctypes as C
import math

import pytest
import torch

NUL, FAKE, ODD = C.c_void_p(0), C.c_void_p(0x1000), C.c_void_p(0x1008)
BIG = 1 << 40


@pytest.fixture(scope="module")
def kvc():
    from eviction_kvc_score_gb300 import build
    build.build()
    from eviction_kvc_score_gb300 import kvc
    return kvc


def cache(kvc, **kw):
    c = kvc.cache(64, 16, 64, 8, "bf16")
    for name, x in kw.items():
        setattr(c, name, x)
    return c


def append(kvc, c, bits=4, table=FAKE, n=4, counts=FAKE, row=FAKE, step=1, k=FAKE, v=FAKE, rows=9, kp=FAKE, vp=FAKE, state=FAKE, size=BIG):
    return kvc._lib.kvc_pages_append_quant(C.byref(c), bits, table, FAKE, n, counts, row, step, k, v, rows, kp, vp, state, size, NUL)


def compact(kvc, c, bits=4, table=FAKE, n=4, idx=FAKE, k_max=3, counts=FAKE, kp=FAKE, vp=FAKE, state=FAKE, size=BIG):
    return kvc._lib.kvc_pages_compact_quant(C.byref(c), bits, table, FAKE, n, idx, k_max, counts, kp, vp, state, size, NUL)


def read(kvc, c, bits=4, table=FAKE, n=4, first=NUL, counts=FAKE, row=FAKE, step=1, kp=FAKE, vp=FAKE, k=FAKE, v=FAKE, rows=9, state=FAKE,
         size=BIG):
    return kvc._lib.kvc_pages_read_quant(C.byref(c), bits, table, FAKE, n, first, counts, row, step, kp, vp, k, v, rows, state, size, NUL)


def attend(kvc, c, bits=4, hq=8, h=2, b=1, m=1, n=4, q=FAKE, qs=512, start=FAKE, table=FAKE, kp=FAKE, vp=FAKE, scale=0.1, out=FAKE,
           ws=FAKE, size=BIG):
    return kvc._lib.kvc_attend_quant(C.byref(c), bits, hq, h, b, m, n, q, qs, start, table, FAKE, kp, vp, scale, out, NUL, ws, size, NUL)


CALLS = dict(kvc_pages_append_quant=append, kvc_pages_compact_quant=compact, kvc_pages_read_quant=read, kvc_attend_quant=attend)


@pytest.mark.parametrize("name", CALLS)
def test_bits_and_caches(kvc, name):
    call = CALLS[name]
    for bits in (0, 1, 2, 3, 5, 7, 16, -4, 1 << 20):
        assert call(kvc, cache(kvc), bits=bits) == -1
        assert "bits" in kvc.kvc_last_error() and name in kvc.kvc_last_error()
    for bad in (dict(n_pages=0), dict(page_rows=8), dict(page_rows=48), dict(head_dim=4), dict(head_dim=68), dict(head_dim=264),
                dict(max_pages=0), dict(max_pages=1 << 27), dict(dtype=2), dict(dtype=-1)):
        assert call(kvc, cache(kvc, **bad)) == -1, bad
        assert name in kvc.kvc_last_error()


def test_rows_arguments(kvc):
    c = cache(kvc)
    for bad in (dict(table=NUL), dict(n=0), dict(n=(1 << 20) + 1), dict(counts=NUL), dict(row=NUL), dict(step=-1), dict(k=NUL),
                dict(v=ODD), dict(rows=-1), dict(kp=ODD), dict(vp=NUL)):
        assert append(kvc, c, **bad) == -1, bad
    for bad in (dict(table=NUL), dict(idx=NUL), dict(k_max=0), dict(counts=NUL), dict(kp=NUL), dict(vp=ODD)):
        assert compact(kvc, c, **bad) == -1, bad
    for bad in (dict(table=NUL), dict(n=0), dict(counts=NUL), dict(row=NUL), dict(step=-1), dict(k=ODD), dict(kp=NUL), dict(vp=NUL),
                dict(k=NUL, v=NUL), dict(rows=-1), dict(vp=ODD)):
        assert read(kvc, c, **bad) == -1, bad
    for call in (append, compact, read):
        for bad in (dict(state=NUL), dict(state=C.c_void_p(0x1010)), dict(size=256)):
            assert call(kvc, c, **bad) == -5, bad


def test_attend_arguments(kvc):
    c = cache(kvc)
    for bad in (dict(hq=7), dict(h=0), dict(b=0), dict(b=1 << 20), dict(m=0), dict(m=1 << 29), dict(n=-1), dict(n=1 << 31), dict(q=NUL),
                dict(q=ODD), dict(qs=504), dict(qs=513), dict(start=NUL), dict(table=NUL), dict(kp=ODD), dict(vp=NUL), dict(out=NUL),
                dict(scale=math.inf), dict(scale=math.nan)):
        assert attend(kvc, c, **bad) == -1, bad
        assert "kvc_attend_quant" in kvc.kvc_last_error()
    assert attend(kvc, c, n=0, q=NUL) == 0
    p = C.byref(c)
    size = kvc._lib.kvc_attend_quant_workspace_size
    assert size(p, 5, 8, 2, 1, 1) == 0 and size(p, 4, 8, 3, 1, 1) == 0 and size(p, 4, 8, 2, 0, 1) == 0
    with pytest.raises(kvc.KvcError):
        kvc.kvc_attend_quant_workspace_size(c, 3, 8, 2, 1, 1)


def test_page_sizes(kvc):
    for bits, d, ps, want in ((4, 128, 16, 16 * 72), (8, 128, 128, 128 * 136), (4, 80, 32, 32 * 54), (8, 8, 16, 16 * 34), (4, 256, 64, 64 * 144)):
        assert kvc.kvc_quant_page_size(kvc.cache(4, ps, d, 4, "f32"), bits) == want
    with pytest.raises(kvc.KvcError):
        kvc.kvc_quant_page_size(cache(kvc), 6)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_quant_page_size(cache(kvc, page_rows=24), 4)


def test_without_a_device_calls_end_with_an_error(kvc):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    for name, call in CALLS.items():
        assert call(kvc, cache(kvc)) == -3
        assert name in kvc.kvc_last_error()


def test_binding_refuses_wrong_tensors(kvc):
    c = cache(kvc)
    i = torch.zeros(4, dtype=torch.int32)
    table, x, pool = torch.zeros((4, 8), dtype=torch.int32), torch.zeros((9, 64), dtype=torch.bfloat16), torch.zeros(64 * 16 * 36, dtype=torch.uint8)
    for call in (lambda: kvc.kvc_pages_append_quant(c, 4, table, i, i, i.long(), 1, x, x, pool, pool, pool),
                 lambda: kvc.kvc_pages_compact_quant(c, 4, table, i, table, i, pool, pool, pool),
                 lambda: kvc.kvc_pages_read_quant(c, 4, table, i, None, i, i.long(), 1, pool, pool, x, x, pool),
                 lambda: kvc.kvc_attend_quant(c, 4, x.view(9, 1, 64), torch.tensor([0, 9], dtype=torch.int32), table, i, pool, pool, 9, x, pool)):
        with pytest.raises(ValueError):    # tensors of the host
            call()


@pytest.mark.parametrize("flags", [2, 3, 1 << 31])
def test_attend_refuses_unknown_flags(kvc, flags):
    c = cache(kvc)
    assert kvc._lib.kvc_attend_quant_ex(C.byref(c), 4, 8, 2, 1, 1, 4, FAKE, 512, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, NUL, flags, FAKE,
                                        BIG, NUL) == -1
    assert "flags" in kvc.kvc_last_error() and "kvc_attend_quant" in kvc.kvc_last_error()
