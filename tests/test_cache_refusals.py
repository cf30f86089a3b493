"""CPU checks of what the paged cache's calls refuse."""
import ctypes as C

import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("bad", ["fp32", "f16", "float16", "", "F32", None, True, 1.0, torch.float16, torch.int32])
def test_types_the_library_does_not_have_are_refused(kvc, bad):
    with pytest.raises(ValueError):
        kvc.cache(64, 16, 64, 8, bad)
    with pytest.raises(ValueError):
        kvc.shape(1, 2, 1, 64, 100, 4, bad)


@pytest.mark.parametrize("code", [2, -1])
def test_unknown_codes_are_refused(kvc, code):
    with pytest.raises(ValueError):
        kvc.cache(64, 16, 64, 8, code)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_workspace_size(kvc.shape(1, 2, 1, 64, 100, 4, code))


@pytest.mark.parametrize("code,names", [(0, ["f32", "float32", torch.float32, 0, np.int32(0)]), (1, ["bf16", "bfloat16", torch.bfloat16, 1, np.int64(1)])])
def test_types_by_every_name(kvc, code, names):
    for name in names:
        assert kvc.cache(64, 16, 64, 8, name).dtype == code
        assert kvc.shape(1, 2, 1, 64, 100, 4, name).dtype == code
