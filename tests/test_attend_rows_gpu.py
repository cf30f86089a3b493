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
    return ((c.out.double() - want).abs() / (tol + 1e-30))[real].max().item()


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


def aim(c, probes, strength=40.0):
    """Row r of list i gets a key along token t's query, so that its logit is about `strength`, the others'
    below half of that: probes are (list, row, token).  All query heads of a token are alike."""
    g = torch.Generator(device="cuda").manual_seed(len(probes))
    n, hq, d = c.q.shape
    c.q.copy_((torch.randint(0, 2, (n, 1, d), generator=g, device="cuda") * 2 - 1).expand(n, hq, d))
    c.kp.mul_(0.1)
    ps = c.kp.shape[1]
    at = torch.tensor(probes, device="cuda")
    page = c.table[at[:, 0], at[:, 1] // ps].long()
    key = torch.zeros((len(probes), d), device="cuda")
    add = c.q[at[:, 2], 0].float() * strength / math.sqrt(d)
    where, same = torch.unique(page * ps + at[:, 1] % ps, return_inverse=True)
    key = torch.zeros((len(where), d), device="cuda").index_add_(0, same, add)
    c.kp.view(-1, d)[where] = key.to(c.kp.dtype)


@pytest.mark.parametrize("dtype,d,hq,ps", [("f32", 64, 2, 16), ("f32", 80, 8, 32), ("bf16", 64, 4, 16), ("bf16", 128, 32, 128),
                                           ("bf16", 96, 2, 64)])
def test_one_row_decides_a_single_token(dtype, d, hq, ps):
    """Lists of 4,000-20,000 rows cut at many places, in each list another row far above the others:
    at the ends, around multiples of 16 to 256, and spread evenly over the whole list, cuts included."""
    lens = [4000 + 1000 * (i % 17) + 13 * i for i in range(40)]
    edges = [m + e for m in (16, 64, 128, 256, 1024, 2048) for e in (-1, 0)]
    c = Case(ns=[1] * 40, lens=lens, hq=hq, h=1, d=d, ps=ps, dtype=dtype, seed=d)
    key = c.kp.clone()
    for shot in range(6):
        rows = []
        for i, t in enumerate(lens):
            k = shot * 40 + i
            rows.append(0 if k == 0 else t - 1 if k % 10 == 0 else edges[k % len(edges)] if k % 3 == 0 else t - edges[k % len(edges)] if k % 3 == 1
                        else int(t * ((0.37 + k * 0.6180339887498949) % 1.0)))
        c.kp.copy_(key)
        aim(c, [(i, r, i) for i, r in enumerate(rows)])
        c.run().check()
        where = c.table[torch.arange(40, device="cuda"), torch.tensor(rows, device="cuda") // ps].long() * ps + torch.tensor(rows, device="cuda") % ps
        assert ((c.out - c.vp.view(-1, d)[where][:, None]).abs() <= 0.02 * c.vp.view(-1, d)[where][:, None].abs() + 1e-3).all()


@pytest.mark.parametrize("dtype,d,hq,h,ns,lens", [
    ("f32", 64, 4, 2, [130, 1, 70], [[130, 900], [300, 1], [70, 513]]), ("f32", 128, 2, 2, [300], [[1000, 300]]),
    ("bf16", 64, 4, 2, [130, 1, 70], [[130, 900], [300, 1], [70, 513]]), ("bf16", 128, 16, 2, [300, 40], [[1000, 300], [77, 40]]),
    ("bf16", 128, 3, 1, [260], [2000]), ("bf16", 80, 4, 1, [130], [400])])
def test_every_token_sees_its_own_row_and_not_the_next(dtype, d, hq, h, ns, lens):
    """Token i's last visible row has a key along its own query and along the token's before it: that
    one may not see the row, or half of its output is another row's."""
    lens = [x for row in lens for x in row] if isinstance(lens[0], list) else lens
    c = Case(ns=ns, lens=lens, hq=hq, h=h, d=d, ps=16, dtype=dtype, seed=d + hq)
    probes = []
    for b, n in enumerate(ns):
        for j in range(h):
            size = c.lens[b * h + j]
            for t in range(n):
                if size - n + t >= 0:
                    probes += [(b * h + j, size - n + t, c.start[b] + t)] + ([(b * h + j, size - n + t, c.start[b] + t - 1)] if t else [])
    aim(c, probes)
    c.run().check()


@pytest.mark.parametrize("d,hq,n", [(64, 2, 1), (80, 16, 4), (128, 3, 40)])
def test_fp32_errors_of_long_lists_stay_small(d, hq, n):
    """Each of T additions rounds a partial sum, whose square grows evenly to the output's: together
    u sqrt(T / 6) of the outputs' root mean square.  Logits of some 5 add 5 * 2^-23 and ex2's 2^-22 to each weight,
    which average out alike.  Four times that is allowed, 1.4e-5; weights of 8 bits would give 2^-9 / sqrt(3), 1.1e-3."""
    t = 20000
    c = Case(ns=[n], lens=[t], hq=hq, h=1, d=d, ps=64, dtype="f32", seed=n)
    c.run()
    torch.cuda.synchronize()
    want, lse, _, _ = ref.attend(c.q, c.start, c.table, c.lens, c.kp, c.vp, c.scale)
    rms = lambda x: x.double().square().mean().sqrt().item()  # noqa: E731
    assert rms(c.out.double() - want) <= 4 * 2.0 ** -24 * math.sqrt(t / 6) * rms(want)
    # the sum has positive terms only: u T / 64 and 64 within the tiles at most, on lse itself
    assert (c.lse.double() - lse).abs().max().item() <= (t / 64 + 64) * 2.0 ** -24 + 16 * 2.0 ** -24 * lse.abs().max().item() + 2.0 ** -20


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 80)])
@pytest.mark.parametrize("most,starts", [
    (40, [-5, 30, 60, 90]), (40, [0, 20, 10, 50]), (40, [3, 30, 300, 310]), (40, [0, 90, 90, 95]), (300, [-2 ** 31, 280, 290, 2 ** 31 - 1]),
    (300, [10, 290, 5, 100]), (300, [400, 200, 100, 50]), (1, [0, 1, 5, 6])])
def test_ranges_of_tokens_are_cut_as_described(dtype, d, most, starts):
    """q_start cut to [0, n_tokens) and max_new: what is left gets its outputs (where it is one sequence's alone),
    everything else keeps what it held, rows before and behind the outputs too."""
    n_tok, hq, h, lens = 320, 4, 2, [350, 40, 10, 500, 77, 300]
    c = Case(ns=[most, 0, n_tok - most], lens=lens, hq=hq, h=h, d=d, ps=16, dtype=dtype, seed=most)
    c.max_new = most
    kvc, guard = K(), 64
    ws = torch.empty(kvc.kvc_attend_workspace_size(c.c, hq, h, 3, most), dtype=torch.uint8, device="cuda")
    kvc.kvc_workspace_init(ws)
    c.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
    out = torch.full((n_tok + 2 * guard, hq, d), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((n_tok + 2 * guard, hq), 7.0, device="cuda")
    c.run(out=out[guard:-guard], lse=lse[guard:-guard], ws=ws)
    torch.cuda.synchronize()
    assert kvc.kvc_workspace_status(ws) == 0x20
    ranges = []
    for a, b in zip(starts, starts[1:]):
        a = max(a, 0)
        ranges.append((a, max(a, min(b, a + most, n_tok))))
    claims = torch.zeros(n_tok + 2 * guard, device="cuda")
    ok = torch.zeros(n_tok, dtype=torch.bool, device="cuda")
    for s, (a, b) in enumerate(ranges):
        if a >= b:
            continue
        # the sequence by itself, its tokens in place
        want, wlse, reach, _ = ref.attend(c.q, [a, b], c.table[s * h:(s + 1) * h], c.lens[s * h:(s + 1) * h], c.kp, c.vp, c.scale)
        tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -16) * reach[a:b] + want[a:b].abs() * torch.finfo(c.q.dtype).eps
        near = ((out[guard + a:guard + b].double() - want[a:b]).abs() <= tol).all(-1).all(-1)
        fine = wlse[a:b].isfinite()
        near &= (((lse[guard + a:guard + b] - wlse[a:b]).abs() <= 1e-4) | ~fine).all(-1)
        ok[a:b] = near
        claims[guard + a:guard + b] += 1
    assert bool(ok[claims[guard:-guard] == 1].all()) and (out[claims == 0] == 7).all() and (lse[claims == 0] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,power", [(1, 24), (1, 40), (1, 117), (300, 28), (300, 40), (300, 117)])
def test_huge_logits(n, d, power):
    """One row has all of the weight: logits beyond 2^24, where product and difference in one step are not the
    difference of the rounded product."""
    c = Case(ns=[n], lens=[1000 + n], hq=4, h=2, d=d, ps=16, dtype="bf16", seed=d + n)
    c.q.mul_(2.0 ** power)
    assert c.q.isfinite().all()
    c.run().check()
