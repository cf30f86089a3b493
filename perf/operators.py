"""Cases, plain forms and calls of the paged-cache operators: rotary positions,
page moves of a compressed cache, and attention of new tokens over it.

A cache here is a pool of pages; a page holds `page` consecutive cached rows of
ONE KV head, and a list is the page-table row of one (layer, sequence, KV head).
Lists have lengths of their own because the budgets of the compression differ
from layer to layer and, optionally, from head to head.
"""
import math

import torch

own = False

F = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step's queries and keys, 64 sequences at far positions: launch latency
        dict(name="rope_decode", op="rope", tokens=64, q_heads=32, k_heads=8, dim=128, rot=128, dtype="bf16",
             interleaved=False, inverse=False, in_place=True, scaled=True, fused=True, pos_hi=131072),
        # a 32K prompt's queries and keys
        dict(name="rope_prompt", op="rope", tokens=32768, q_heads=32, k_heads=8, dim=128, rot=128, dtype="bf16",
             interleaved=False, inverse=False, in_place=False, scaled=True, fused=False, pos_hi=32768),
        # kept keys taken back to position zero: interleaved pairs in half of an odd head size, fp32
        dict(name="rope_partial_f32", op="rope", tokens=4099, q_heads=0, k_heads=12, dim=80, rot=40, dtype="f32",
             interleaved=True, inverse=True, in_place=False, scaled=False, fused=False, pos_hi=1000000),
        # five draft tokens of 16 sequences, after the last ones were rolled back
        dict(name="pages_draft", op="pages", kind="draft", layers=1, seqs=16, heads=8, dim=128, page=16, dtype="bf16",
             len_lo=200, len_hi=2300, rows_lo=5, rows_hi=5, fan=0),
        # the compressed 32-layer prompt put into pages, per-list row counts
        dict(name="pages_prompt", op="pages", kind="prompt", layers=32, seqs=1, heads=8, dim=128, page=64, dtype="bf16",
             len_lo=0, len_hi=0, rows_lo=384, rows_hi=4000, fan=0),
        # a running cache forked and its copy evicted to a quarter
        dict(name="pages_evict", op="pages", kind="evict", layers=8, seqs=4, heads=8, dim=128, page=32, dtype="bf16",
             len_lo=1500, len_hi=6000, rows_lo=400, rows_hi=1500, fan=1),
        # eight continuations of each of four sequences take one token each: shared last pages are copied
        dict(name="pages_beams_f32", op="pages", kind="beams", layers=2, seqs=4, heads=4, dim=64, page=16, dtype="f32",
             len_lo=100, len_hi=900, rows_lo=1, rows_hi=1, fan=8),
        # the next token of one short sequence: launch latency
        dict(name="attend_decode_one", op="attend", seqs=1, q_heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             n_lo=1, n_hi=1, len_lo=900, len_hi=1100),
        # the next token of 64 sequences over compressed lists
        dict(name="attend_decode_batch", op="attend", seqs=64, q_heads=32, kv_heads=8, dim=128, page=16, dtype="bf16",
             n_lo=1, n_hi=1, len_lo=500, len_hi=6000),
        # draft tokens over a few long lists, head size 64
        dict(name="attend_draft_long", op="attend", seqs=3, q_heads=16, kv_heads=4, dim=64, page=128, dtype="bf16",
             n_lo=3, n_hi=7, len_lo=60000, len_hi=131000),
        # chunks of several prompts, fp32, an odd head size
        dict(name="attend_chunk_f32", op="attend", seqs=5, q_heads=8, kv_heads=8, dim=80, page=32, dtype="f32",
             n_lo=1, n_hi=301, len_lo=0, len_hi=2500),
        # one long chunk behind a long cache
        dict(name="attend_chunk_long", op="attend", seqs=1, q_heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             n_lo=4096, n_hi=4096, len_lo=28672, len_hi=28672),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "pages", "attend", "attend"])
    if op == "rope":
        dim = rng.choice([32, 64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        k = rng.choice([1, 2, 4, 8, 12])
        q = k * rng.choice([0, 1, 4, 5])
        most = 32768 * 40 * 128 // ((q + k) * dim)
        return dict(op=op, tokens=_log(rng, 1, min(most // 2, 50000)), q_heads=q, k_heads=k, dim=dim, rot=rot,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.3, in_place=rng.random() < 0.5, scaled=rng.random() < 0.5,
                    fused=rng.random() < 0.5 and q > 0, pos_hi=_log(rng, 2, 1 << 20))
    if op == "pages":
        kind = rng.choice(["draft", "prompt", "evict", "beams"])
        seqs, layers = _log(rng, 1, 12), _log(rng, 1, 6)
        hi = _log(rng, 20, 3000)
        rows = {"draft": 7, "prompt": 2000, "evict": max(1, hi // 3), "beams": 2}[kind]
        r = _log(rng, 1, rows)
        return dict(op=op, kind=kind, layers=layers, seqs=seqs, heads=rng.choice([1, 2, 4, 5, 8]),
                    dim=rng.choice([64, 80, 128]), page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), len_lo=rng.randint(0, hi), len_hi=hi,
                    rows_lo=rng.randint(0, r), rows_hi=r, fan={"evict": 1, "beams": rng.randint(1, 6)}.get(kind, 0))
    kv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128, 80 if dtype == "f32" else 64])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    seqs = _log(rng, 1, 40)
    n_hi = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 1200)])
    # tokens x keys x heads stays below the longest chunk's, fp32 below a thirtieth of it
    most = int((1.2e9 if dtype == "bf16" else 4e7) / (seqs * n_hi * kv * group) * 128 / dim)
    hi = _log(rng, 1, max(2, min(most, 100000, 4000000 // (seqs * kv))))
    return dict(op="attend", seqs=seqs, q_heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                dtype=dtype, n_lo=rng.randint(1, n_hi), n_hi=n_hi, len_lo=rng.randint(0, hi), len_hi=hi)


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], uneven but the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ rotary positions

SCALED = dict(factor=8.0, alpha=1.0, beta=4.0, context=8192)


def _frequencies(rot, scaled, theta=500000.0):
    """Radians per position of every pair; scaled: pairs that turn fewer than alpha times in the trained context are
    slowed down by the factor, those that turn beta times or more are kept, with a linear blend between."""
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if scaled:
        turns = SCALED["context"] * f / (2 * math.pi)
        keep = ((turns - SCALED["alpha"]) / (SCALED["beta"] - SCALED["alpha"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / SCALED["factor"])
    return f


def _prepare_rope(c, g):
    q, k, d, n = c["q_heads"], c["k_heads"], c["dim"], c["tokens"]
    dt = F[c["dtype"]]
    # fused: queries, keys and values of a token side by side, as one projection leaves them
    width = (q + 2 * k) * d
    s = dict(case=c, pos=torch.randint(0, c["pos_hi"], (n,), generator=g, device="cuda", dtype=torch.int32))
    if c["fused"]:
        x = torch.randn((n, width), generator=g, device="cuda").to(dt)
        s["q"], s["k"] = x[:, :q * d].view(n, q, d), x[:, q * d:(q + k) * d].view(n, k, d)
        s["x"] = x
    else:
        s["q"] = torch.randn((n, q, d), generator=g, device="cuda").to(dt) if q else None
        s["k"] = torch.randn((n, k, d), generator=g, device="cuda").to(dt)
    if c["in_place"]:
        s["q_out"], s["k_out"] = s["q"], s["k"]
    else:
        s["q_out"] = torch.empty((n, q, d), device="cuda", dtype=dt) if q else None
        s["k_out"] = torch.empty((n, k, d), device="cuda", dtype=dt)
    s["freq"] = _frequencies(c["rot"], c["scaled"])
    if own:
        from eviction_kvc_score_gb300 import kvc
        s["table"] = torch.empty(c["rot"] // 2, device="cuda", dtype=torch.int64)
        kvc.kvc_rope_table(c["rot"], 500000.0, s["table"], **(SCALED if c["scaled"] else {}))
    return s


def _rotate(x, cos, sin, rot, interleaved):
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _run_rope(s):
    c = s["case"]
    if own:
        from eviction_kvc_score_gb300 import kvc
        kvc.kvc_rope(s["table"], s["pos"], s["q"], s["k"], s["q_out"], s["k_out"], c["rot"],
                     interleaved=c["interleaved"], inverse=c["inverse"])
    else:
        angle = (s["pos"].double()[:, None] * s["freq"])[:, None]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        sin = -sin if c["inverse"] else sin
        if s["q"] is not None:
            s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]))
        s["k_out"].copy_(_rotate(s["k"], cos, sin, c["rot"], c["interleaved"]))
    # the fused rows come back whole: the values beside the keys stay as they were
    return s["x"] if c["fused"] and c["in_place"] else [s["q_out"], s["k_out"]] if s["q"] is not None else s["k_out"]


def _exact_rope(c, seed):
    s = _prepare_rope(c, _generator(seed))
    angle = s["pos"].double()[:, None] * s["freq"]
    turn = torch.complex(torch.cos(angle), -torch.sin(angle) if c["inverse"] else torch.sin(angle))[:, None]
    done = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        y, r = x.double().clone(), c["rot"]
        if c["interleaved"]:
            y[..., :r] = torch.view_as_real(torch.view_as_complex(y[..., :r].reshape(*y.shape[:2], r // 2, 2).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * turn
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        done.append(y)
    if c["fused"] and c["in_place"]:
        n, d = c["tokens"], c["dim"]
        return torch.cat([y.reshape(n, -1) for y in done] + [s["x"][:, (c["q_heads"] + c["k_heads"]) * d:].double()], 1)
    return done if s["q"] is not None else done[0]


# ------------------------------------------------------------------ pages

def _page_sizes(c):
    """Lengths before the pass and rows per list, the number of lists that hold them, of all lists, and of pages."""
    held = c["layers"] * c["seqs"] * c["heads"]
    lists = held * (1 + c["fan"])
    base = [0] * held if c["kind"] == "prompt" else _spread(held, c["len_lo"], c["len_hi"])
    base += [0] * (lists - held)
    took = lists if c["fan"] == 0 else lists - held
    rows = _spread(took, c["rows_lo"], c["rows_hi"])
    if c["kind"] == "evict":
        rows = [min(r, base[i % held]) for i, r in enumerate(rows)]
    most = max(base) + max(rows)
    used = sum(_up(b, c["page"]) for b in base)
    fresh = sum(_up(r, c["page"]) + 1 for r in rows)
    return base, rows, held, lists, _up(most, c["page"]) + 1, used + fresh + 64


def _prepare_pages(c, g):
    base, rows, held, lists, width, n_pages = _page_sizes(c)
    ps, d, dt = c["page"], c["dim"], F[c["dtype"]]
    i32 = dict(device="cuda", dtype=torch.int32)
    s = dict(case=c, held=held)
    s["k_pool"] = torch.randn((n_pages, ps, d), generator=g, device="cuda").to(dt)
    s["v_pool"] = torch.randn((n_pages, ps, d), generator=g, device="cuda").to(dt)
    s["table"] = torch.full((lists, width), -1, **i32)
    s["len"] = torch.zeros(lists, **i32)
    s["base"] = torch.tensor(base, **i32)
    # the rows that the lists hold at the start, then those of the pass
    n = sum(base)
    first = torch.randn((2, max(n, 1), d), generator=g, device="cuda").to(dt)
    start = torch.cumsum(s["base"].long(), 0) - s["base"]
    _make_handle(s, n_pages, lists)
    _append(s, s["base"], start, 1, first[0], first[1])
    count = [0] * (lists - len(rows)) + rows
    s["count"] = torch.tensor(count, **i32)
    if c["kind"] == "evict":
        s["count"][:held] = -1
        # the kept rows' positions, ascending, one random row in each stretch of the list
        k = max(1, max(rows))
        parent = torch.arange(lists, device="cuda") % held
        span = (s["base"][parent] / s["count"].clamp(min=1)).double()[:, None]
        at = torch.arange(k, device="cuda") + torch.rand((lists, k), generator=g, device="cuda", dtype=torch.float64)
        s["idx"] = torch.minimum((at * span).long(), (s["base"][parent].long() - 1).clamp(min=0)[:, None]).int()
    else:
        m = max(1, sum(rows))
        s["new"] = torch.randn((2, m, d), generator=g, device="cuda").to(dt)
        if c["kind"] == "prompt":   # packed rows, list after list
            s["row"], s["step"] = torch.cumsum(s["count"].long(), 0) - s["count"], 1
        else:                       # token-major rows: [sequence][token][head] of each layer
            s["step"] = c["heads"]
            h = torch.arange(lists, device="cuda") % c["heads"]
            group = torch.arange(lists, device="cuda") // c["heads"]
            widest = s["count"].view(-1, c["heads"]).amax(1).long()
            s["row"] = (torch.cumsum(widest, 0) - widest)[group] * c["heads"] + h
            s["new"] = torch.randn((2, max(1, int(widest.sum())) * c["heads"], d), generator=g, device="cuda").to(dt)
    if c["fan"]:
        # list held + j * held + i continues list i
        s["src"] = torch.cat([torch.full((held,), -1, **i32), torch.arange(held, **i32).repeat(c["fan"])])
        s["keep"] = torch.cat([torch.full((held,), -1, **i32), torch.zeros(lists - held, **i32)])
    else:
        s["keep"] = s["base"].clone()
    return s


def _make_handle(s, n_pages, lists):
    c = s["case"]
    if own:
        from eviction_kvc_score_gb300 import kvc
        s["cache"] = kvc.cache(n_pages, c["page"], c["dim"], s["table"].shape[1], c["dtype"])
        s["state"] = torch.empty(kvc.kvc_pages_size(s["cache"], lists), device="cuda", dtype=torch.uint8)
        kvc.kvc_pages_init(s["cache"], s["state"])
    else:
        s["refs"] = torch.zeros(n_pages, device="cuda", dtype=torch.int32)


def _parts(n):
    """For counts n: the owner and the place within it of every element."""
    n = n.long()
    who = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n)
    return who, torch.arange(who.numel(), device=n.device) - (torch.cumsum(n, 0) - n)[who]


def _take(s, need):
    """The lowest free pages, for lists that need so many each: owner, place within the owner, page."""
    who, at = _parts(need)
    page = torch.nonzero(s["refs"] == 0).view(-1)[:who.numel()]
    s["refs"][page] = 1
    return who, at, page.int()


def _drop(s, who, at):
    page = s["table"][who, at].long()
    s["refs"].index_add_(0, page, torch.full_like(page, -1, dtype=torch.int32))


def _move(s, dst, k, v, src):
    d = s["case"]["dim"]
    s["k_pool"].view(-1, d)[dst] = k.view(-1, d)[src]
    s["v_pool"].view(-1, d)[dst] = v.view(-1, d)[src]


def _append(s, count, row, step, k, v):
    """count[i] rows, row[i] + r * step of k and v, behind list i; a shared last page is copied first."""
    if own:
        from eviction_kvc_score_gb300 import kvc
        kvc.kvc_pages_append(s["cache"], s["table"], s["len"], count, row, step, k, v, s["k_pool"], s["v_pool"], s["state"])
        return
    ps, t = s["case"]["page"], s["table"]
    old = s["len"].long()
    count = count.long()
    had, has = (old + ps - 1) // ps, (old + count + ps - 1) // ps
    every = torch.arange(old.numel(), device="cuda")
    last = t[every, (old // ps).clamp(max=t.shape[1] - 1)]
    shared = (old % ps > 0) & (count > 0) & (s["refs"][last.clamp(min=0).long()] > 1)
    who, at, page = _take(s, (has - had + shared.long()) * (count > 0))
    t[who, (had - shared.long())[who] + at] = page
    s["refs"].index_add_(0, last[shared].long(), torch.full((int(shared.sum()),), -1, device="cuda", dtype=torch.int32))
    who, at = _parts((old % ps) * shared)
    _move(s, t[who, old[who] // ps].long() * ps + at, s["k_pool"], s["v_pool"], last[who].long() * ps + at)
    who, at = _parts(count)
    to = old[who] + at
    _move(s, t[who, to // ps].long() * ps + to % ps, k, v, row[who] + at * step)
    s["len"].add_(count.int())


def _truncate(s, keep):
    if own:
        from eviction_kvc_score_gb300 import kvc
        kvc.kvc_pages_truncate(s["cache"], s["table"], s["len"], keep, s["state"])
        return
    ps = s["case"]["page"]
    new = torch.where(keep >= 0, torch.minimum(keep, s["len"]), s["len"])
    has, had = (new + ps - 1) // ps, (s["len"] + ps - 1) // ps
    who, at = _parts(had - has)
    _drop(s, who, has[who] + at)
    s["len"].copy_(new)


def _fork(s, src):
    if own:
        from eviction_kvc_score_gb300 import kvc
        kvc.kvc_pages_fork(s["cache"], s["table"], s["len"], src, s["state"])
        return
    ps = s["case"]["page"]
    n = torch.where(src >= 0, s["len"][src.clamp(min=0).long()], 0)
    who, at = _parts((n + ps - 1) // ps)
    page = s["table"][src[who].long(), at]
    s["table"][who, at] = page
    s["refs"].index_add_(0, page.long(), torch.ones_like(page))
    s["len"].add_(n)


def _compact(s, idx, count):
    if own:
        from eviction_kvc_score_gb300 import kvc
        kvc.kvc_pages_compact(s["cache"], s["table"], s["len"], idx, count, s["k_pool"], s["v_pool"], s["state"])
        return
    ps, old = s["case"]["page"], s["table"].clone()
    n = count.clamp(min=0)
    who, at, page = _take(s, (n + ps - 1) // ps)
    to = torch.full_like(old, -1)
    to[who, at] = page
    who, at = _parts(n)
    src = idx[who, at].long()
    _move(s, to[who, at // ps].long() * ps + at % ps, s["k_pool"], s["v_pool"], old[who, src // ps].long() * ps + src % ps)
    who, at = _parts(torch.where(count >= 0, (s["len"] + ps - 1) // ps, 0))
    _drop(s, who, at)
    s["table"].copy_(torch.where(to >= 0, to, old))
    s["len"].copy_(torch.where(count >= 0, count, s["len"]))


def _run_pages(s):
    kind = s["case"]["kind"]
    _truncate(s, s["keep"])   # what the pass before added goes back to the pool
    if s["case"]["fan"]:
        _fork(s, s["src"])
    if kind == "evict":
        _compact(s, s["idx"], s["count"])
    else:
        _append(s, s["count"], s["row"], s["step"], s["new"][0], s["new"][1])
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"], "table": s["table"], "len": s["len"]}


# ------------------------------------------------------------------ attention

def _attend_sizes(c):
    n = _spread(c["seqs"], c["n_lo"], c["n_hi"])
    lens = [x + n[i // c["kv_heads"]] for i, x in enumerate(_spread(c["seqs"] * c["kv_heads"], c["len_lo"], c["len_hi"]))]
    return n, lens


def _prepare_attend(c, g):
    n, lens = _attend_sizes(c)
    ps, d, b, h, dt = c["page"], c["dim"], c["seqs"], c["kv_heads"], F[c["dtype"]]
    i32 = dict(device="cuda", dtype=torch.int32)
    pages = [_up(x, ps) for x in lens]
    n_pages, width = sum(pages) + 5, max(pages) + 1
    s = dict(case=c, max_new=max(n), len=torch.tensor(lens, **i32))
    s["q_start"] = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), **i32)
    # keys with a few strong channels, as real ones have; pages in no order
    k = torch.randn((n_pages, ps, d), generator=g, device="cuda")
    k[..., torch.randperm(d, generator=g, device="cuda")[:4]] *= 3
    s["k_pool"] = k.to(dt)
    s["v_pool"] = torch.randn((n_pages, ps, d), generator=g, device="cuda").to(dt)
    s["q"] = torch.randn((sum(n), c["q_heads"], d), generator=g, device="cuda").to(dt)
    who, at = _parts(torch.tensor(pages, device="cuda"))
    s["table"] = torch.full((b * h, width), -1, **i32)
    s["table"][who, at] = torch.randperm(n_pages, generator=g, device="cuda")[:who.numel()].int()
    if own:
        from eviction_kvc_score_gb300 import kvc
        s["cache"] = kvc.cache(n_pages, ps, d, width, c["dtype"])
        s["ws"] = torch.empty(kvc.kvc_attend_workspace_size(s["cache"], c["q_heads"], h, b, s["max_new"]), device="cuda", dtype=torch.uint8)
        kvc.kvc_workspace_init(s["ws"])
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    return s


def _run_attend(s):
    c = s["case"]
    if own:
        from eviction_kvc_score_gb300 import kvc
        kvc.kvc_attend(s["cache"], s["q"], s["q_start"], s["table"], s["len"], s["k_pool"], s["v_pool"],
                       s["max_new"], s["out"], s["ws"], lse=s["lse"])
        return [s["out"], s["lse"]]
    b, h, d, ps = c["seqs"], c["kv_heads"], c["dim"], c["page"]
    g, m = c["q_heads"] // h, s["max_new"]
    t = (s["table"].shape[1] - 1) * ps
    key = torch.arange(t, device="cuda")
    row = s["table"].view(b, h, -1)[:, :, key // ps].clamp(min=0).long() * ps + key % ps
    n = s["q_start"][1:] - s["q_start"][:-1]
    token = torch.arange(m, device="cuda")
    at = (s["q_start"][:-1, None] + token).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"].float()[at].view(b, m, h, g, d).permute(0, 2, 3, 1, 4).reshape(b, h, g * m, d)
    score = q @ s["k_pool"].view(-1, d)[row].float().transpose(-1, -2)
    score.mul_(1 / math.sqrt(d))
    # token i of n sees the first len - n + i + 1 keys of its list
    sees = (s["len"].view(b, h, 1) - n[:, None, None] + token + 1)[:, :, None, :, None] > key
    score = score.view(b, h, g, m, t).masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, h, g * m, t) @ s["v_pool"].view(-1, d)[row].float()).view(b, h, g, m, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    real = (token < n[:, None])
    o = o.permute(0, 3, 1, 2, 4)[real].reshape(s["q"].shape).to(s["q"].dtype)
    return [o, lse.permute(0, 3, 1, 2, 4)[real].reshape(s["q"].shape[:2]).contiguous()]


def _exact_attend(c, seed):
    s = _prepare_attend(c, _generator(seed))
    n, lens = _attend_sizes(c)
    h, g, ps, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["page"], c["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for i in range(c["seqs"]):
        for j in range(h):
            size = lens[i * h + j]
            pages = s["table"][i * h + j, :_up(size, ps)].long()
            k = s["k_pool"][pages].reshape(-1, d)[:size].double()
            v = s["v_pool"][pages].reshape(-1, d)[:size].double()
            for u in range(0, n[i], 1024):
                w = min(n[i], u + 1024)
                x = s["q"][first + u:first + w, j * g:(j + 1) * g].double()
                z = torch.einsum("ngd,td->ngt", x, k) / math.sqrt(d)
                last = size - n[i] + torch.arange(u, w, device="cuda")
                z = z.masked_fill(torch.arange(size, device="cuda") > last[:, None, None], -math.inf)
                out[first + u:first + w, j * g:(j + 1) * g] = torch.einsum("ngt,td->ngd", torch.softmax(z, -1), v)
                lse[first + u:first + w, j * g:(j + 1) * g] = torch.logsumexp(z, -1)
        first += n[i]
    return [out, lse]


# ------------------------------------------------------------------ all of them

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def prepare(case, seed):
    make = {"rope": _prepare_rope, "pages": _prepare_pages, "attend": _prepare_attend}[case["op"]]
    return make(dict(case), _generator(seed))


def run(state):
    return {"rope": _run_rope, "pages": _run_pages, "attend": _run_attend}[state["case"]["op"]](state)


def exact(case, seed):
    if case["op"] == "pages":
        return None   # rows are moved, not computed
    return (_exact_rope if case["op"] == "rope" else _exact_attend)(dict(case), seed)


def work(case):
    c, size = case, 4 if case["dtype"] == "f32" else 2
    if c["op"] == "rope":
        x = c["tokens"] * (c["q_heads"] + c["k_heads"]) * (c["rot"] if c["in_place"] else c["dim"])
        return {"bytes": 2 * x * size + 4 * c["tokens"] + 4 * c["rot"],
                "flops": 3 * c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["rot"]}
    if c["op"] == "pages":
        base, rows, held, lists, width, _ = _page_sizes(c)
        ps, moved = c["page"], sum(rows)
        entries = sum(_up(r, ps) for r in rows)
        if c["fan"]:
            entries += c["fan"] * 2 * sum(_up(b, ps) for b in base)
        if c["kind"] == "beams":   # the shared rows of last pages
            moved += sum(base[i % held] % ps for i, r in enumerate(rows) if r)
        return {"bytes": 4 * moved * c["dim"] * size + 4 * entries + 16 * lists + (4 * moved if c["kind"] == "evict" else 0), "flops": 0}
    n, lens = _attend_sizes(c)
    h, g = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    pairs = sum(m * x - m * (m - 1) // 2 for x, m in ((x, n[i // h]) for i, x in enumerate(lens)))
    moved = 2 * sum(lens) * c["dim"] + 2 * sum(n) * c["q_heads"] * c["dim"]
    return {"bytes": moved * size + 4 * sum(n) * c["q_heads"] + 4 * sum(_up(x, c["page"]) for x in lens),
            "flops": 4 * pairs * g * c["dim"]}
