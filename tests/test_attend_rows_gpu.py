"""Attention over the paged cache, row by row: what lies behind lists and in
memory that a tile used before, single rows that decide the whole output, and
errors that do not grow with a list's length."""
import math

import pytest
import torch

import cache_ref as ref
from test_attend_gpu import Case, K

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


def worst(c, weights):
    """Largest |error| / tolerance of the outputs; weights: error of a probability relative to it."""
    torch.cuda.synchronize()
    want, lse, reach, logit = ref.attend(c.q, c.start, c.table, c.lens, c.kp, c.vp, c.scale)
    u, d = 2.0 ** -24, c.q.shape[-1]
    # the terms of test_attend_gpu, and twice the probabilities' error (they are summed unrounded)
    dx = 2 * (d + 4) * u * logit + 4 * u * logit + 2.0 ** -21
    tol = (2 * dx + 2 * (max(c.lens) + 64) * u + 2 * weights)[..., None] * reach + want.abs() * torch.finfo(c.q.dtype).eps / 2 * 1.001
    real = ~want.isnan()
    return ((c.out.double() - want).abs() / tol)[real].max().item()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ns,lens,hq", [([1, 1, 3], [1, 900, 300], 8), ([130, 40], [700, 40], 8), ([300], [300], 2)])
def test_probabilities_keep_sixteen_bits(ns, lens, hq, d):
    """The tensor cores get each probability as two bf16 numbers: the upper 8 bits, cut off, and what
    is left, rounded to 8 bits: 2^-7 2^-9 of it at most."""
    c = Case(ns=ns, lens=lens, hq=hq, h=2, d=d, ps=32, dtype="bf16", seed=d + hq)
    assert worst(c.run(), 2.0 ** -16) <= 1


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 300])
@pytest.mark.parametrize("flat", [False, True])
def test_infinite_values_of_rows_that_every_token_sees(d, n, flat):
    """They reach the outputs, in their columns alone; also where every probability is a power of two,
    whose second term is nothing."""
    c = Case(ns=[n], lens=[1000 + n], hq=4, h=2, d=d, ps=16, dtype="bf16", seed=d + n)
    if flat:
        c.q.zero_()
    page = c.table[0, 200 // 16].item()
    c.vp[page, 200 % 16, 3] = math.inf
    c.vp[page, 200 % 16, 5] = -math.inf
    c.vp[c.table[0, 40].item(), 2, 6] = math.nan
    c.run()
    torch.cuda.synchronize()
    assert (c.out[:, :2, 3] == math.inf).all() and (c.out[:, :2, 5] == -math.inf).all()
    assert c.out[:, :2, 6].isnan().all()
    c.out[:, :2, 3:7] = 0
    assert c.out.isfinite().all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 80), ("f32", 64)])
@pytest.mark.parametrize("ns", [[1, 5], [200, 1]])
def test_one_bf16_probability_is_the_callers_choice(dtype, d, ns):
    """On the tensor cores 2^-8 of a probability may be lost then; on the CUDA cores nothing changes."""
    c = Case(ns=ns, lens=[700, 300], hq=4, h=2, d=d, ps=32, dtype=dtype, seed=d)
    c.run()
    out, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(7)
    K().kvc_attend_ex(c.c, c.q, c.q_start, c.table, c.len, c.kp, c.vp, c.max_new, c.out, K().ATTEND_BF16_P, c.ws,
                      lse=c.lse, scale=c.scale)
    c.check()
    tc = dtype == "bf16" and d != 80
    assert torch.equal(c.lse, lse) and torch.equal(c.out, out) != tc
    if tc:      # and the one is nearer to the definition
        want = ref.attend(c.q, c.start, c.table, c.lens, c.kp, c.vp, c.scale)[0]
        assert (c.out.double() - want).norm() > 1.1 * (out.double() - want).norm()
