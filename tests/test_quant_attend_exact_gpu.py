"""How exact attention over a cache held in 4 or 8 bits is, beyond the bound per
element of test_quant_attend_gpu.py: the error's norm, channels that are zero, and rows
that some tokens do not see."""
import math

import pytest
import torch

import quant_ref as ref
from test_quant_attend_gpu import Case, K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


# Each form of the call: one token, drafts (units of 16 and 32 rows), chunks, single tokens
# beside a chunk, head sizes of every kernel.
FORMS = [
    dict(ns=[1, 1], lens=[700, 2300], hq=8, h=2, d=128, ps=16),
    dict(ns=[1], lens=[30000], hq=4, h=2, d=64, ps=64),
    dict(ns=[4, 3], lens=[500, 1800], hq=8, h=2, d=128, ps=32),
    dict(ns=[7, 5], lens=[1500, 300], hq=8, h=2, d=64, ps=128),
    dict(ns=[8], lens=[900], hq=8, h=2, d=128, ps=32),
    dict(ns=[1], lens=[900], hq=64, h=1, d=128, ps=32),
    dict(ns=[90, 200], lens=[1500, 300], hq=4, h=2, d=128, ps=64),
    dict(ns=[150], lens=[4000], hq=6, h=2, d=64, ps=16),
    dict(ns=[1, 70, 1], lens=[1200, 900, 40], hq=8, h=2, d=128, ps=16),
    dict(ns=[1, 3], lens=[300, 800], hq=4, h=2, d=80, ps=16),
    dict(ns=[40, 90], lens=[1000, 300], hq=4, h=2, d=96, ps=32),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_channels_that_are_zero_stay_zero(i, dtype, bits):
    """V's channels 3, 32 and the last are 0 in every row, in groups whose other values
    lie to one side of zero or to both: (n - z) s is 0, and so are the outputs, exactly."""
    d = FORMS[i]["d"]
    zero = [3, 32, d - 1]

    def change(k, v):
        for j, x in enumerate(v):
            if j % 2:
                x.sub_(4)
            x[:, zero] = 0
    c = Case(**FORMS[i], dtype=dtype, bits=bits, seed=i, change=change)
    assert any(ref.quantise(x, bits)[2][:, zero].amax() > 0 for x in c.v)
    c.run().check()
    assert (c.out[..., zero] == 0).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_errors_norm(i, dtype, bits):
    c = Case(**FORMS[i], dtype=dtype, bits=bits, seed=100 + i).run()
    torch.cuda.synchronize()
    want = ref.attend(c.q, c.start, c.k, c.v, c.scale, bits)["out"]
    assert ref.near(c.out, want) is None


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 80), ("f32", 128)])
@pytest.mark.parametrize("ns", [[4, 3], [8, 2], [12, 9], [70, 200]])
def test_values_that_a_token_does_not_see_leave_no_trace(ns, dtype, d, bits):
    """The last token's own row of V is 2^40 to 2^99 times as large as the others, in one group of channels or
    in all: the tokens before it get the very bits that they get without it."""
    c = Case(ns=ns, lens=[[300, 777], [129, 1000]], hq=8, h=2, d=d, ps=16, dtype=dtype, bits=bits)
    c.run().check()
    calm = c.out.clone(), c.lse.clone()

    def change(k, v):
        v[0][-1] *= 2.0 ** 40
        v[1][-1, :32] = 2.0 ** 99
        v[2][-1, 32:] *= -(2.0 ** 60)
        v[3][-1, 5] = 2.0 ** 45
    c = Case(ns=ns, lens=[[300, 777], [129, 1000]], hq=8, h=2, d=d, ps=16, dtype=dtype, bits=bits, change=change)
    c.run()
    torch.cuda.synchronize()
    before = [t for t in range(sum(ns)) if t + 1 not in c.start]
    assert len(before) > 3
    assert torch.equal(c.out[before], calm[0][before]) and torch.equal(c.lse, calm[1])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 80), ("f32", 128)])
@pytest.mark.parametrize("ns", [[1, 1], [8, 5], [70, 90]])
def test_rows_small_in_value_and_probability_keep_their_bits(ns, dtype, d, bits):
    """Channels 32 to 63 of V are 2^-30 of the others and half of the rows have 2^-25 of the others' probability (their
    values, 2^25 times as large there, decide those channels as much as the likely rows do): their outputs are as near to
    the definition as anybody's."""
    def change(k, v):
        for x, y in zip(k, v):
            x.copy_(torch.randn_like(x.float()) / 64)
            x[::2, 0], x[1::2, 0] = 8, -8
            y[:, 32:64] *= 2.0 ** -30
            y[1::2, 32:64] *= 2.0 ** 25
    c = Case(ns=ns, lens=[500, 900], hq=8, h=2, d=d, ps=32, dtype=dtype, bits=bits, change=change)
    c.q[..., 0] = 1.08 * math.sqrt(d)    # logits of +-8.64: e^-17.3 between the halves
    c.run()
    torch.cuda.synchronize()
    want = ref.attend(c.q, c.start, c.k, c.v, c.scale, bits)["out"]
    assert ref.near(c.out[..., 32:64], want[..., 32:64], logit=8.64) is None


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 80), ("f32", 64)])
@pytest.mark.parametrize("ns", [[1, 3], [200, 60]])
def test_one_bf16_probability_is_the_callers_choice(dtype, d, ns, bits):
    """In tcgen05's kernel 2^-8 of a probability may be lost then; in the others nothing changes."""
    c = Case(ns=ns, lens=[700, 300], hq=4, h=2, d=d, ps=32, dtype=dtype, bits=bits, seed=d)
    c.run()
    out, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(7)
    K().kvc_attend_quant_ex(c.c, bits, c.q, c.q_start, c.table, c.len, c.kp, c.vp, c.max_new, c.out, K().ATTEND_BF16_P, c.ws,
                            lse=c.lse, scale=c.scale)
    torch.cuda.synchronize()
    one = dtype == "bf16" and d != 80 and ns[0] > 16
    assert torch.equal(c.lse, lse) and torch.equal(c.out, out) != one
    if one:
        r = ref.attend(c.q, c.start, c.k, c.v, c.scale, bits)
        # both sums' weights move by the logits' error (as in Case.check); p is rounded to nearest, the output once more
        dx = (2 * (d + 18) * r["logit_w"] + 2.0 ** 3) * 2.0 ** -24
        tol = (2 * dx[..., None] + 2.0 ** -9 + 2.0 ** -14) * r["reach"] + 2.0 ** -9 * r["out"].abs() * 1.01
        assert ((c.out.double() - r["out"]).abs() <= tol).all()
        assert (c.out.double() - r["out"]).norm() > 1.1 * (out.double() - r["out"]).norm()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 96), ("f32", 64)])
@pytest.mark.parametrize("ns", [[1, 1], [6, 4], [70, 40]])
def test_largest_and_smallest_queries(ns, dtype, d, bits):
    """Queries of 2^123 over keys that are 2^-123 of the usual ones or nothing, and the other way round:
    logits are ordinary numbers, and 0 of a row of zeros."""
    tiny = -123 if dtype == "bf16" else -100    # three bf16 pieces end at 2^-133
    for big, small in ((2.0 ** 123, 2.0 ** -123), (2.0 ** tiny, 2.0 ** (-3 - tiny))):
        def change(k, v):
            for x in k:
                x.mul_(small)
                x[3::7] = 0
        c = Case(ns=ns, lens=[300, 170], hq=4, h=2, d=d, ps=16, dtype=dtype, bits=bits, change=change)
        c.q.mul_(big)
        assert c.q.isfinite().all() and all(x.isfinite().all() for x in c.k)
        c.run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,power", [(1, 121), (6, 121), (80, 40), (80, 117)])
def test_huge_queries_over_ordinary_keys(n, d, bits, power):
    """Logits of 2^40 and more: one row has all of the weight.  (tcgen05's sums of products of 3.5 2^121 with strong
    channels of 15 pass 2^128, as they do in fp32: 16 times smaller ones for the lists it takes.)"""
    c = Case(ns=[n], lens=[300], hq=4, h=2, d=d, ps=16, dtype="bf16", bits=bits)
    c.q.mul_(2.0 ** power)
    assert c.q.isfinite().all()
    c.run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d,n", [(128, 1), (64, 3), (128, 4)])
@pytest.mark.parametrize("odd", [2.0 ** 124, math.inf, math.nan])
def test_huge_queries_leave_the_others_alone(odd, d, n, bits):
    """Rows beside a query that is huge or no number get the very bits that they get beside an ordinary one, also over
    keys of 2^110."""
    for size in (1.0, 2.0 ** 110):
        def change(k, v):
            for x in k:
                x.mul_(size)
        c = Case(ns=[n], lens=[300], hq=8, h=2, d=d, ps=16, dtype="bf16", bits=bits, change=change)
        if size > 1:
            c.q.mul_(2.0 ** -108)
        c.run().check()
        out, lse = c.out.clone(), c.lse.clone()
        c.q[0, 2, 5] = odd
        c.run()
        torch.cuda.synchronize()
        others = torch.ones(c.lse.shape, dtype=torch.bool)
        others[0, 2] = False
        assert torch.equal(c.out[others], out[others]) and torch.equal(c.lse[others], lse[others])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(FORMS)))
@pytest.mark.parametrize("power", [100, -100])
def test_largest_and_smallest_values(power, i, dtype, bits):
    """Values up to 2^100, which sums over the longest lists may not pass, all of one sign so that they add up; and
    values of 2^-100."""
    def change(k, v):
        for x, y in zip(k, v):
            x.mul_(0.01)
            y.copy_((torch.rand_like(y.float()) * 0.5 + 0.5).clamp(max=0.99) * 2.0 ** power)
    c = Case(**FORMS[i], dtype=dtype, bits=bits, seed=i, change=change).run()
    c.check()
    want = ref.attend(c.q, c.start, c.k, c.v, c.scale, bits)["out"]
    assert want.abs().max() > 2.0 ** (power - 1) and ref.near(c.out, want) is None


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,d,n", [("bf16", 64, 1), ("bf16", 128, 8), ("f32", 64, 1), ("bf16", 80, 1)])
def test_large_values_of_lists_that_one_block_adds_up(dtype, d, n, bits):
    """So many lists that a list is one block's, of 131,072 rows each with values of up to 2^100, alike and all of them seen
    alike: the outputs are their mean.  (All lists are the same pages.)"""
    lists, rows = 600, 131072

    def change(k, v):
        k[0].zero_()
        v[0].copy_((torch.rand_like(v[0].float()) * 0.5 + 0.5).clamp(max=0.99) * 2.0 ** 100)
    c = Case(ns=[n], lens=[rows], hq=1, h=1, d=d, ps=128, dtype=dtype, bits=bits, change=change)
    kvc = K()
    q = c.q.repeat(lists, 1, 1)
    q_start = torch.arange(lists + 1, dtype=torch.int32, device="cuda") * n
    ws = torch.empty(kvc.kvc_attend_quant_workspace_size(c.c, bits, 1, 1, lists, n), dtype=torch.uint8, device="cuda")
    kvc.kvc_workspace_init(ws)
    out = torch.full_like(q, 7.0)
    kvc.kvc_attend_quant(c.c, bits, q, q_start, c.table.repeat(lists, 1), c.len.repeat(lists), c.kp, c.vp, n, out, ws)
    torch.cuda.synchronize()
    assert kvc.kvc_workspace_status(ws) == 0
    v = ref.stands(c.v[0], bits).cumsum(0)
    want = torch.stack([v[rows - n + t] / (rows - n + t + 1) for t in range(n)])[:, None].repeat(lists, 1, 1)
    # T positive terms, added up by 128 or more partial sums; the output rounded once
    assert ((out.double() - want).abs() <= want * (2 * (rows / 128 + 64) * 2.0 ** -24 + torch.finfo(out.dtype).eps / 2)).all()
