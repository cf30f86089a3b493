"""A wait of the attention kernel that runs out.  With KVC_TEST_SKIP_ARRIVE=1
every block leaves its first load out, so a stage is never filled and the
bounded waits on it expire: the call records KVC_DEV_TIMEOUT, ends within
seconds and leaves the context usable -- after the workspace is initialised
again, the next call gives what the call before gave."""
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


@pytest.mark.parametrize("n,length", [(1, 900), (200, 900)])
def test_missing_load_times_out_and_context_recovers(monkeypatch, n, length):
    from eviction_kvc_score_gb300 import kvc
    g = torch.Generator(device="cuda").manual_seed(1)
    pages = -(-length // 64)
    c = kvc.cache(2 * pages, 64, 128, pages, "bf16")
    kp = torch.randn((2 * pages, 64, 128), generator=g, device="cuda").bfloat16()
    vp = torch.randn((2 * pages, 64, 128), generator=g, device="cuda").bfloat16()
    table = torch.arange(2 * pages, device="cuda", dtype=torch.int32).view(2, pages)
    lens = torch.full((2,), length, device="cuda", dtype=torch.int32)
    q = torch.randn((n, 8, 128), generator=g, device="cuda").bfloat16()
    start = torch.tensor([0, n], device="cuda", dtype=torch.int32)
    ws = torch.empty(kvc.kvc_attend_workspace_size(c, 8, 2, 1, n), dtype=torch.uint8, device="cuda")
    kvc.kvc_workspace_init(ws)

    def run():
        out = torch.zeros_like(q)
        kvc.kvc_attend(c, q, start, table, lens, kp, vp, n, out, ws)
        torch.cuda.synchronize()
        return out
    good = run()
    assert kvc.kvc_workspace_status(ws) == 0
    monkeypatch.setenv("KVC_TEST_SKIP_ARRIVE", "1")
    t0 = time.time()
    run()
    assert time.time() - t0 < 30.0
    assert kvc.kvc_workspace_status(ws) & kvc.DEV_TIMEOUT
    monkeypatch.delenv("KVC_TEST_SKIP_ARRIVE")
    kvc.kvc_workspace_init(ws)
    assert torch.equal(run(), good)
    assert kvc.kvc_workspace_status(ws) == 0
