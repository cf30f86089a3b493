"""The operators of a cache held in 4 or 8 bits together, as a program that answers
from a compressed prompt uses them: score, budget and compact a prompt, quantise the
packed rows into pages, fork; decode tokens and drafts (rotate, quantise, attend), roll
drafts back, evict one copy, attend over it, read rows back, give everything back."""
import pytest
import torch

import quant_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype,d,bits", [("bf16", 128, 4), ("bf16", 64, 8), ("f32", 64, 4)])
def test_compress_quantise_then_decode(dtype, d, bits):
    from eviction_kvc_score_gb300 import kvc, workloads as wk
    wl = wk.ZIGZAG_32K.scaled(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=d, seq_len=1500, window=32, dtype=dtype,
                              total_budget=2 * 300, layer_floor=40, temperature=None)
    L, HQ, H, T, W, ps = 2, 8, 2, wl.seq_len, wl.window, 32
    dt = wl.torch_dtype
    x = wk.make_inputs(wl, 78, device="cuda")
    total, floor = wl.budget_args()
    b = kvc.alloc_buffers(kvc.shape_of(wl), total, wl.k_max)
    kvc.compress(b, x["q"], x["k"], x["v"], total, floor, wl.mass_num, wl.mass_den)

    seqs, n_pages = 2, 400   # sequence 0 holds the prompt; 1 is its fork
    c = kvc.cache(n_pages, ps, d, 100, dtype)
    lists, per = L * seqs * H, seqs * H
    table = torch.full((lists, c.max_pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(lists, dtype=torch.int32, device="cuda")
    # NaN wherever nothing is written
    kp, vp = (torch.full((n_pages, kvc.kvc_quant_page_size(c, bits)), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    state = torch.empty(kvc.kvc_pages_size(c, lists), dtype=torch.uint8, device="cuda")
    kvc.kvc_pages_init(c, state)

    # the packed rows, without a copy of the budgets to the host
    rows = (b.budget.clamp(0, T - W) + W).repeat_interleave(H).view(L, H)
    start = (rows.flatten().cumsum(0) - rows.flatten()).view(L, H)
    counts = torch.zeros((L, seqs, H), dtype=torch.int32, device="cuda")
    counts[:, 0] = rows
    src_row = torch.zeros((L, seqs, H), dtype=torch.int64, device="cuda")
    src_row[:, 0] = start
    kvc.kvc_pages_append_quant(c, bits, table, lens, counts.view(-1), src_row.view(-1), 1, b.k_out, b.v_out, kp, vp, state)
    src = torch.full((L, seqs, H), -1, dtype=torch.int32, device="cuda")
    src[:, 1] = (torch.arange(L, device="cuda")[:, None] * seqs * H + torch.arange(H, device="cuda")).int()
    kvc.kvc_pages_fork(c, table, lens, src.view(-1), state)

    rot = torch.empty(d // 2, dtype=torch.int64, device="cuda")
    kvc.kvc_rope_table(d, 500000.0, rot, factor=8.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    # the rows of each list as they were handed over
    hold = [[o[start[l, h]:start[l, h] + rows[l, h]].clone() for o in (b.k_out, b.v_out)]
            for l in range(L) for _ in range(seqs) for h in range(H)]

    def read_back():
        n = lens.tolist()
        assert n == [pair[0].shape[0] for pair in hold]
        at = lens.long().cumsum(0) - lens
        out = [torch.full((sum(n), d), 7.0, dtype=dt, device="cuda") for _ in range(2)]
        kvc.kvc_pages_read_quant(c, bits, table, lens, None, lens, at, 1, kp, vp, *out, state)
        for got, j in zip(out, (0, 1)):
            assert torch.equal(got.double(), torch.cat([ref.stands(pair[j], bits) for pair in hold]))

    def attend(l, q, n):
        t, ln = table[l * per:(l + 1) * per], lens[l * per:(l + 1) * per]
        q_start = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
        ws = torch.empty(kvc.kvc_attend_quant_workspace_size(c, bits, HQ, H, seqs, n), dtype=torch.uint8, device="cuda")
        kvc.kvc_workspace_init(ws)
        out = torch.empty((seqs * n, HQ, d), dtype=dt, device="cuda")
        kvc.kvc_attend_quant(c, bits, q, q_start, t, ln, kp, vp, n, out, ws)
        k, v = ([hold[l * per + i][j] for i in range(per)] for j in (0, 1))
        r = ref.attend(q, [0, n, 2 * n], k, v, d ** -0.5, bits)
        # a logit's sums, the sums over rows, for bf16 probabilities and steps rounded to
        # fp16 (2^-11 each; 2^-24 half lost per row at 2^6), the output's rounding
        u, size = 2.0 ** -24, max(y.shape[0] for y in k)
        dx = 2 * (d + 18) * u * r["logit_w"] + 2.0 ** -34 * r["logit_top"] + 2.0 ** -21
        tol = 2 * dx[..., None] * r["reach"] + 2 * (size + 64) * u * r["reach_w"]
        if dtype == "bf16":
            tol = tol + 2.0 ** -10 * r["reach_w"] + (size * 2.0 ** -30 + 2.0 ** -23) * ref.N[bits] * r["step"][..., None]
        assert ((out.double() - r["out"]).abs() <= tol + r["out"].abs() * torch.finfo(dt).eps / 2 * 1.001).all()
        assert kvc.kvc_workspace_status(ws) == 0

    read_back()
    pos = T
    for n in (1, 3, 40, 1):               # a token, draft tokens, a chunk, a token
        p = torch.arange(pos, pos + n, dtype=torch.int32, device="cuda").repeat(seqs)
        for l in range(L):
            qkv = torch.randn((seqs * n, (HQ + 2 * H) * d), generator=g, device="cuda").to(dt)
            q, k, v = (y.view(seqs * n, -1, d) for y in qkv.split([HQ * d, H * d, H * d], 1))
            kvc.kvc_rope(rot, p, q, k, q, k, d)
            t, ln = table[l * per:(l + 1) * per], lens[l * per:(l + 1) * per]
            # rows of the fused projection, taken where they lie
            step = HQ + 2 * H
            first = torch.arange(seqs, device="cuda")[:, None] * n * step + HQ + torch.arange(H, device="cuda")
            kvc.kvc_pages_append_quant(c, bits, t, ln, torch.full((per,), n, dtype=torch.int32, device="cuda"), first.view(-1).long(), step,
                                       qkv, qkv.view(-1, d)[H:].contiguous(), kp, vp, state)
            for s in range(seqs):
                for h in range(H):
                    i = l * per + s * H + h
                    hold[i] = [torch.cat([hold[i][0], k[s * n:(s + 1) * n, h]]), torch.cat([hold[i][1], v[s * n:(s + 1) * n, h]])]
            attend(l, q, n)
        if n == 3:                        # the drafts are rolled back
            keep = torch.tensor([pair[0].shape[0] - 3 for pair in hold], dtype=torch.int32, device="cuda")
            kvc.kvc_pages_truncate(c, table, lens, keep, state)
            hold = [[y[:-3] for y in pair] for pair in hold]
        else:
            pos += n
    read_back()

    # the fork is evicted to every second row; the other sequence keeps its own
    m = max(pair[0].shape[0] for pair in hold)
    idx = (torch.arange(m // 2 + 1, device="cuda") * 2).int().repeat(lists, 1)
    counts = torch.full((L, seqs, H), -1, dtype=torch.int32, device="cuda")
    counts[:, 1] = (lens.view(L, seqs, H)[:, 1] + 1) // 2
    kvc.kvc_pages_compact_quant(c, bits, table, lens, idx, counts.view(-1), kp, vp, state)
    hold = [[y[::2] if i // H % seqs else y for y in pair] for i, pair in enumerate(hold)]
    read_back()
    for l in range(L):
        attend(l, torch.randn((seqs, HQ, d), generator=g, device="cuda").to(dt), 1)
    kvc.kvc_pages_truncate(c, table, lens, torch.zeros_like(lens), state)
    assert kvc.kvc_pages_status(c, state) == (0, n_pages)
