"""Attention over the paged cache, row by row: what lies behind lists and in
memory that a tile used before, single rows that decide the whole output, and
errors that do not grow with a list's length."""
import math

import pytest
import torch

import cache_ref as ref
from test_attend_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("d,hq,ps", [(128, 8, 16), (64, 16, 128), (128, 2, 64)])
def test_warps_without_rows_wait_for_their_clean_values(d, hq, ps):
    """Single tokens of few query heads: three of four warps have no rows of
    their own and only take NaN and infinities out of V, behind every list and
    in what a stage held before."""
    lens = [1 + (97 * i * i + 13 * i) % 700 for i in range(192)]
    c = Case(ns=[1] * 96, lens=lens, hq=hq, h=2, d=d, ps=ps, dtype="bf16", seed=d + ps)
    c.run().check()
    out, lse = c.out.clone(), c.lse.clone()
    for again in range(20):
        c.out.fill_(7)
        c.run()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse), again


@pytest.mark.parametrize("dtype,d,hq,n", [("bf16", 128, 8, 1), ("bf16", 64, 2, 5), ("bf16", 128, 64, 3), ("f32", 64, 8, 1)])
def test_joins_read_only_what_this_call_wrote(dtype, d, hq, n):
    """Lists shared by few and by many blocks: what the slots held before is NaN, so a lane that
    reads another block's slot before it may gives NaN."""
    c = Case(ns=[n] * 3, lens=[40000, 9000, 70000], hq=hq, h=1, d=d, ps=64, dtype=dtype, seed=hq)
    c.run().check()
    out, lse = c.out.clone(), c.lse.clone()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    slots = 256 + 16 * 4 * sms * 4      # behind the header and the counters
    for again in range(20):
        c.ws[slots:] = 255
        c.out.fill_(7)
        c.run()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse), again
