"""A wait that runs out in the tensor cores' attention over held rows.  With
KVC_TEST_SKIP_ARRIVE=1 the warps that make tiles say nothing of their first one,
and those that read few rows' keys leave their first load out, so the bounded waits
on it expire: the call records KVC_DEV_TIMEOUT, ends within
seconds and leaves the context usable -- after the workspace is initialised again,
the next call gives what the call before gave."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", [1, 200])
def test_missing_load_times_out_and_context_recovers(monkeypatch, n, bits):
    from test_quant_attend_gpu import Case, K
    kvc = K()
    c = Case(ns=[n], lens=[900], hq=8, h=2, d=128, ps=64, dtype="bf16", bits=bits)

    def run():
        c.out.fill_(7), c.lse.fill_(7)
        c.run()
        torch.cuda.synchronize()
        return c.out.clone()
    good = run()
    c.check()
    monkeypatch.setenv("KVC_TEST_SKIP_ARRIVE", "1")
    t0 = time.time()
    run()
    assert time.time() - t0 < 30.0
    assert kvc.kvc_workspace_status(c.ws) & kvc.DEV_TIMEOUT
    monkeypatch.delenv("KVC_TEST_SKIP_ARRIVE")
    kvc.kvc_workspace_init(c.ws)
    assert torch.equal(run(), good)
    c.check()
