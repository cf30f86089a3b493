"""CPU checks of what the paged cache's calls refuse."""
import ctypes as C

import pytest

NUL, FAKE = C.c_void_p(0), C.c_void_p(0x1000)


@pytest.fixture(scope="module")
def kvc():
    from eviction_kvc_score_gb300 import build
    build.build()
    from eviction_kvc_score_gb300 import kvc
    return kvc


@pytest.mark.parametrize("flags", [2, 3, 1 << 31])
def test_attend_refuses_unknown_flags(kvc, flags):
    c = kvc.cache(64, 16, 64, 8, "bf16")
    assert kvc._lib.kvc_attend_ex(C.byref(c), 8, 2, 1, 1, 4, FAKE, 512, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, NUL,
                                  flags, FAKE, 1 << 40, NUL) == -1
    assert "flags" in kvc.kvc_last_error()
