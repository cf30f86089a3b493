"""The cache operators together, as a program that answers from a compressed
prompt uses them: score, budget and compact a prompt, put the packed rows into
pages, and decode: rotate, append, attend; fork the cache, evict one copy by
its own keys' order, roll drafts back, and give everything back."""
import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_compress_then_decode(dtype, d):
    from eviction_kvc_score_gb300 import kvc, workloads as wk
    wl = wk.ZIGZAG_32K.scaled(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=d, seq_len=1500, window=32, dtype=dtype,
                              total_budget=2 * 300, layer_floor=40, temperature=None)
    L, HQ, H, T, W, ps = 2, 8, 2, wl.seq_len, wl.window, 16
    dt = wl.torch_dtype
    x = wk.make_inputs(wl, 77, device="cuda")
    total, floor = wl.budget_args()
    b = kvc.alloc_buffers(kvc.shape_of(wl), total, wl.k_max)
    kvc.compress(b, x["q"], x["k"], x["v"], total, floor, wl.mass_num, wl.mass_den)

    # sequence 0 holds the prompt; 1 is its fork
    seqs, n_pages = 2, 400
    c = kvc.cache(n_pages, ps, d, 100, dtype)
    lists = L * seqs * H
    table = torch.full((lists, c.max_pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(lists, dtype=torch.int32, device="cuda")
    kp = torch.full((n_pages, ps, d), float("nan"), dtype=dt, device="cuda")
    vp = kp.clone()
    state = torch.empty(kvc.kvc_pages_size(c, lists), dtype=torch.uint8, device="cuda")
    kvc.kvc_pages_init(c, state)

    # the packed rows, without a copy of the budgets to the host
    rows = (b.budget.clamp(0, T - W) + W).repeat_interleave(H).view(L, H)
    start = (rows.flatten().cumsum(0) - rows.flatten()).view(L, H)
    counts = torch.zeros((L, seqs, H), dtype=torch.int32, device="cuda")
    counts[:, 0] = rows
    src_row = torch.zeros((L, seqs, H), dtype=torch.int64, device="cuda")
    src_row[:, 0] = start
    kvc.kvc_pages_append(c, table, lens, counts.view(-1), src_row.view(-1), 1, b.k_out, b.v_out, kp, vp, state)
    src = torch.full((L, seqs, H), -1, dtype=torch.int32, device="cuda")
    src[:, 1] = (torch.arange(L, device="cuda")[:, None] * seqs * H + torch.arange(H, device="cuda")).int()
    kvc.kvc_pages_fork(c, table, lens, src.view(-1), state)

    rot = torch.empty(d // 2, dtype=torch.int64, device="cuda")
    kvc.kvc_rope_table(d, 500000.0, rot, factor=8.0)
    freq = ref.rope_frequencies(d, 500000.0, 8.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    per = seqs * H
    # what each list has to hold, gathered from the packed outputs
    hold = [[b.k_out[start[l, h]:start[l, h] + rows[l, h]].clone(), b.v_out[start[l, h]:start[l, h] + rows[l, h]].clone()]
            for l in range(L) for _ in range(seqs) for h in range(H)]
    pos = T
    for n in (1, 3, 1):                       # a token, three draft tokens, a token
        q_start = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
        p = torch.arange(pos, pos + n, dtype=torch.int32, device="cuda").repeat(seqs)
        for l in range(L):
            qkv = torch.randn((seqs * n, (HQ + 2 * H) * d), generator=g, device="cuda").to(dt)
            q = qkv[:, :HQ * d].view(-1, HQ, d)
            k = qkv[:, HQ * d:(HQ + H) * d].view(-1, H, d)
            v = qkv[:, (HQ + H) * d:].view(-1, H, d)
            k0 = k.clone()
            kvc.kvc_rope(rot, p, q, k, q, k, d)
            want_k = ref.rope(k0, p, freq, False)
            assert (k.double() - want_k).abs().max() <= 2.0 ** -8 * want_k.abs().max() + 1e-5
            t, ln = table[l * per:(l + 1) * per], lens[l * per:(l + 1) * per]
            # rows of the fused projection, taken where they lie
            step = HQ + 2 * H
            head = torch.arange(H, device="cuda")
            first = torch.arange(seqs, device="cuda")[:, None] * n * step + HQ + head
            kvc.kvc_pages_append(c, t, ln, torch.full((per,), n, dtype=torch.int32, device="cuda"), first.view(-1).long(), step,
                                 qkv, qkv.view(-1, d)[H:].contiguous(), kp, vp, state)
            for s in range(seqs):
                for h in range(H):
                    i = l * per + s * H + h
                    hold[i] = [torch.cat([hold[i][0], k[s * n:(s + 1) * n, h]]), torch.cat([hold[i][1], v[s * n:(s + 1) * n, h]])]
            ws = torch.empty(kvc.kvc_attend_workspace_size(c, HQ, H, seqs, n), dtype=torch.uint8, device="cuda")
            kvc.kvc_workspace_init(ws)
            out = torch.empty((seqs * n, HQ, d), dtype=dt, device="cuda")
            kvc.kvc_attend(c, q, q_start, t, ln, kp, vp, n, out, ws)
            size = [hold[l * per + i][0].shape[0] for i in range(per)]
            assert ln.tolist() == size
            # the definition on the rows as they were handed over
            pool_k, pool_v = (torch.cat([hold[l * per + i][j] for i in range(per)]) for j in (0, 1))
            at = torch.tensor([0] + size).cumsum(0)
            flat_k, flat_v = torch.zeros((per, max(size), d), dtype=dt, device="cuda"), torch.zeros((per, max(size), d), dtype=dt, device="cuda")
            for i in range(per):
                flat_k[i, :size[i]], flat_v[i, :size[i]] = pool_k[at[i]:at[i + 1]], pool_v[at[i]:at[i + 1]]
            want, _, reach, logit = ref.attend(q, [0, n, 2 * n], torch.arange(per, device="cuda")[:, None], size, flat_k, flat_v, d ** -0.5)
            u = 2.0 ** -24
            dx = 2 * (d + 6) * u * logit + 2.0 ** -21
            tol = (2 * dx + 2 * (max(size) + 64) * u + (2.0 ** -8 if dtype == "bf16" else 0))[..., None] * reach
            assert ((out.double() - want).abs() <= tol + want.abs() * torch.finfo(dt).eps / 2 * 1.001).all()
            assert kvc.kvc_workspace_status(ws) == 0
        if n == 3:                            # the drafts are rolled back
            keep = torch.tensor([x[0].shape[0] - 3 for x in hold], dtype=torch.int32, device="cuda")
            kvc.kvc_pages_truncate(c, table, lens, keep, state)
            hold = [[x[:-3] for x in pair] for pair in hold]
        else:
            pos += n

    # the fork is evicted to every second row; the other sequence keeps its own
    m = max(x[0].shape[0] for x in hold)
    idx = (torch.arange(m // 2 + 1, device="cuda") * 2).int().repeat(lists, 1)
    counts = torch.full((L, seqs, H), -1, dtype=torch.int32, device="cuda")
    counts[:, 1] = (lens.view(L, seqs, H)[:, 1] + 1) // 2
    kvc.kvc_pages_compact(c, table, lens, idx, counts.view(-1), kp, vp, state)
    for i, pair in enumerate(hold):
        step = 2 if i // H % seqs else 1
        size = lens[i].item()
        pages = table[i, :-(-size // ps)].long()
        for pool, want in zip((kp, vp), pair):
            assert torch.equal(pool[pages].view(-1, d)[:size], want[::step])
    kvc.kvc_pages_truncate(c, table, lens, torch.zeros_like(lens), state)
    assert kvc.kvc_pages_status(c, state) == (0, n_pages)
