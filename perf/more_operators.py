"""Cases, plain forms and calls of the operators on a paged cache held in 4 or 8 bits: rows quantised as they are
written, moved and read back, and attention of new tokens over them.

A row of K or V is held in groups of 32 channels, the last one filled up with zeros. A group of values x has codes n of
b bits, a step s and a zero code z, and stands for (n - z) s:
  s = (max(x, 0) - min(x, 0)) / (2^b - 1), rounded up to four significant bits (b = 4) or to a power of two (b = 8);
  z = -min(x, 0) / s and n = x / s + z, to the nearest.
The step before it is rounded up, and the factor 1 / s, are rounded to 32 bits: that is the format, not an inaccuracy.
"""
import math

import torch

own = False

F = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step's keys and values of 16 sequences, written and read back: launch latency
        dict(name="quant4_token", op="quant", kind="token", bits=4, layers=1, seqs=16, heads=8, dim=128, page=16, dtype="bf16",
             len_lo=200, len_hi=2300, rows_lo=1, rows_hi=1),
        # the compressed 32-layer prompt put into pages in 4 bits, per-list row counts, and read back
        dict(name="quant4_prompt", op="quant", kind="prompt", bits=4, layers=32, seqs=1, heads=8, dim=128, page=64, dtype="bf16",
             len_lo=0, len_hi=0, rows_lo=384, rows_hi=4000),
        # chunks of several prompts in fp32 at an odd head size, token-major
        dict(name="quant8_chunk_f32", op="quant", kind="token", bits=8, layers=2, seqs=5, heads=4, dim=80, page=32, dtype="f32",
             len_lo=0, len_hi=700, rows_lo=30, rows_hi=520),
        # the rows of long lists taken back out of 8 bits
        dict(name="quant8_read", op="quant", kind="read", bits=8, layers=4, seqs=2, heads=8, dim=128, page=128, dtype="bf16",
             len_lo=3000, len_hi=16000, rows_lo=2900, rows_hi=2900),
        # a running 4-bit cache forked and its copy evicted to a quarter
        dict(name="quant4_evict", op="quant", kind="evict", bits=4, layers=8, seqs=4, heads=8, dim=128, page=32, dtype="bf16",
             len_lo=1500, len_hi=6000, rows_lo=400, rows_hi=1500),
        # the next token of one short sequence: launch latency
        dict(name="attend4_one", op="attend", bits=4, seqs=1, q_heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             n_lo=1, n_hi=1, len_lo=900, len_hi=1100),
        # the next token of 64 sequences over compressed lists
        dict(name="attend4_batch", op="attend", bits=4, seqs=64, q_heads=32, kv_heads=8, dim=128, page=16, dtype="bf16",
             n_lo=1, n_hi=1, len_lo=500, len_hi=6000),
        # the same in 8 bits, half as many
        dict(name="attend8_batch", op="attend", bits=8, seqs=32, q_heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             n_lo=1, n_hi=1, len_lo=500, len_hi=6000),
        # draft tokens over a few long lists, head size 64
        dict(name="attend4_draft_long", op="attend", bits=4, seqs=3, q_heads=16, kv_heads=4, dim=64, page=128, dtype="bf16",
             n_lo=3, n_hi=7, len_lo=60000, len_hi=131000),
        # chunks of several prompts, fp32, an odd head size
        dict(name="attend4_chunk_f32", op="attend", bits=4, seqs=5, q_heads=8, kv_heads=8, dim=80, page=32, dtype="f32",
             n_lo=1, n_hi=301, len_lo=0, len_hi=2500),
        # chunks of several prompts, some of them short, over 8 bits
        dict(name="attend8_chunks", op="attend", bits=8, seqs=6, q_heads=32, kv_heads=8, dim=128, page=32, dtype="bf16",
             n_lo=1, n_hi=700, len_lo=0, len_hi=5000),
        # one long chunk behind a long cache
        dict(name="attend4_chunk_long", op="attend", bits=4, seqs=1, q_heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
             n_lo=4096, n_hi=4096, len_lo=28672, len_hi=28672),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, bits = rng.choice(["quant", "attend", "attend"]), rng.choice([4, 4, 8])
    if op == "quant":
        kind = rng.choice(["token", "prompt", "read", "evict"])
        seqs, layers, hi = _log(rng, 1, 12), _log(rng, 1, 6), _log(rng, 20, 3000)
        r = _log(rng, 1, {"token": 600, "prompt": 2000, "read": 3000, "evict": max(1, hi // 3)}[kind])
        return dict(op=op, kind=kind, bits=bits, layers=layers, seqs=seqs, heads=rng.choice([1, 2, 4, 5, 8]),
                    dim=rng.choice([32, 64, 80, 96, 128, 128, 192, 256]), page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), len_lo=rng.randint(0, hi), len_hi=hi,
                    rows_lo=rng.randint(0, r), rows_hi=r)
    kv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128, 80 if dtype == "f32" else 64])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    seqs = _log(rng, 1, 40)
    n_hi = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 1200)])
    # tokens x keys x heads stays below the longest chunk's, fp32 below a thirtieth of it
    most = int((1.2e9 if dtype == "bf16" else 4e7) / (seqs * n_hi * kv * group) * 128 / dim)
    hi = _log(rng, 1, max(2, min(most, 100000, 4000000 // (seqs * kv))))
    return dict(op="attend", bits=bits, seqs=seqs, q_heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                dtype=dtype, n_lo=rng.randint(1, n_hi), n_hi=n_hi, len_lo=rng.randint(0, hi), len_hi=hi)


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], uneven but the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _up(a, b):
    return -(-a // b)


def _starts(n):
    """Where each of consecutive runs of n elements begins."""
    return torch.cumsum(n.long(), 0) - n.long()


def _parts(n):
    """For counts n: the owner and the place within it of every element."""
    n = n.long()
    who = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n)
    return who, torch.arange(who.numel(), device=n.device) - _starts(n)[who]


def _rows(g, n, d, dt, strong):
    """n rows of d channels; keys have a few strong channels, as real ones do, off zero by several of their deviations."""
    x = torch.randn((max(n, 1), d), generator=g, device="cuda")
    if strong:
        at = torch.randperm(d, generator=g, device="cuda")[:4]
        x[:, at] = 3 * x[:, at] + 8
    return x.to(dt)


# ------------------------------------------------------------------ the format, in elementary operations

def _quantise(x, bits):
    """Codes [rows][groups][32], steps and zero codes [rows][groups] of x [rows][channels]."""
    rows, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -d % 32)).view(rows, _up(d, 32), 32)
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    most = 2 ** bits - 1
    step = (hi * 0.5 - lo * 0.5) / torch.full_like(hi, most / 2)
    drop = 20 if bits == 4 else 23   # bits of the 23 that are rounded up
    step = ((step.view(torch.int32) + ((1 << drop) - 1)) >> drop << drop).view(torch.float32).clamp(min=2.0 ** -126)
    inv = torch.ones_like(step) / step
    zero = torch.round(-lo * inv)
    code = (torch.round(x * inv[..., None]) + zero[..., None]).clamp(0, most)
    step = torch.where((x.abs() < 2.0 ** 126).all(-1), step, math.nan)
    return code.to(torch.uint8), step, zero.to(torch.uint8)


def _values(code, step, zero, d):
    return ((code.float() - zero.float()[..., None]) * step[..., None]).flatten(-2)[..., :d]


# ------------------------------------------------------------------ rows written, moved and read back

def _quant_sizes(c):
    """Lengths before the pass and rows of every list, and how many lists the pass works on."""
    held = c["layers"] * c["seqs"] * c["heads"]
    base = [0] * held if c["kind"] == "prompt" else _spread(held, c["len_lo"], c["len_hi"])
    if c["kind"] == "token":   # all heads of a layer's sequence take the same tokens
        rows = [r for r in _spread(held // c["heads"], c["rows_lo"], c["rows_hi"]) for _ in range(c["heads"])]
    else:
        rows = _spread(held, c["rows_lo"], c["rows_hi"])
        if c["kind"] != "prompt":
            rows = [min(r, b) for r, b in zip(rows, base)]
    return base, rows, held


def _prepare_quant(c, g):
    base, rows, held = _quant_sizes(c)
    d, dt, kind, bits = c["dim"], F[c["dtype"]], c["kind"], c["bits"]
    i32 = dict(device="cuda", dtype=torch.int32)
    s = dict(case=c, held=held, base=torch.tensor(base, **i32), count=torch.tensor(rows, **i32))
    first = [_rows(g, sum(base), d, dt, strong) for strong in (True, False)]
    s["out"] = [torch.empty((max(1, sum(rows)), d), device="cuda", dtype=dt) for _ in range(2)]
    s["to"] = _starts(s["count"])
    if kind == "token":     # token-major rows: [sequence][token][head] of each layer
        h = c["heads"]
        s["step"] = h
        s["row"] = _starts(s["count"][::h]).repeat_interleave(h) * h + torch.arange(held, device="cuda") % h
    else:                   # packed rows, list after list
        s["step"], s["row"] = 1, s["to"]
    if kind in ("token", "prompt"):
        s["new"] = [_rows(g, sum(rows), d, dt, strong) for strong in (True, False)]
    if kind == "evict":
        # the kept rows' positions, ascending, one random row in each stretch of the list
        span = (s["base"] / s["count"].clamp(min=1)).double()[:, None]
        k = max(1, max(rows))
        at = torch.arange(k, device="cuda") + torch.rand((held, k), generator=g, device="cuda", dtype=torch.float64)
        s["idx"] = torch.minimum((at * span).long(), (s["base"].long() - 1).clamp(min=0)[:, None]).int()
    # read: rows from somewhere inside the list
    s["from"] = (s["base"] - s["count"]) // 2 if kind == "read" else torch.zeros_like(s["base"]) if kind == "evict" else s["base"]
    if own:
        from eviction_kvc_score_gb300 import kvc
        ps, lists = c["page"], held * (2 if kind == "evict" else 1)
        n_pages = sum(_up(b, ps) + _up(r, ps) + 1 for b, r in zip(base, rows)) + 64
        s["cache"] = kvc.cache(n_pages, ps, d, _up(max(base) + max(rows), ps) + 1, c["dtype"])
        s["state"] = torch.empty(kvc.kvc_pages_size(s["cache"], lists), device="cuda", dtype=torch.uint8)
        kvc.kvc_pages_init(s["cache"], s["state"])
        size = kvc.kvc_quant_page_size(s["cache"], bits)
        s["pool"] = [torch.zeros((n_pages, size), device="cuda", dtype=torch.uint8) for _ in range(2)]
        s["table"] = torch.full((lists, s["cache"].max_pages), -1, **i32)
        s["len"] = torch.zeros(lists, **i32)
        kvc.kvc_pages_append_quant(s["cache"], bits, s["table"][:held], s["len"][:held], s["base"], _starts(s["base"]), 1, *first,
                                   *s["pool"], s["state"])
        if kind == "evict":   # list held + i continues list i
            s["src"] = torch.cat([torch.full((held,), -1, **i32), torch.arange(held, **i32)])
            s["keep"] = torch.cat([torch.full((held,), -1, **i32), torch.zeros(held, **i32)])
            s["idx"], s["every"] = s["idx"].repeat(2, 1), torch.cat([torch.full((held,), -1, **i32), s["count"]])
    else:
        # each list's rows stand together, with room behind them for the pass's
        s["start"] = _starts(s["base"] + s["count"])
        who, at = _parts(s["base"])
        slots = max(1, sum(base) + sum(rows))
        s["held_rows"] = []
        for x in first:
            parts = _quantise(x[:sum(base)], bits)
            room = [torch.zeros((slots, *p.shape[1:]), device="cuda", dtype=p.dtype) for p in parts]
            for p, r in zip(parts, room):
                r[s["start"][who] + at] = p
            s["held_rows"].append(room)
        s["len"] = s["base"].clone()
    return s


def _run_quant_own(s):
    from eviction_kvc_score_gb300 import kvc
    c, bits, kind = s["cache"], s["case"]["bits"], s["case"]["kind"]
    table, lens = s["table"], s["len"]
    if kind == "evict":
        kvc.kvc_pages_truncate(c, table, lens, s["keep"], s["state"])
        kvc.kvc_pages_fork(c, table, lens, s["src"], s["state"])
        kvc.kvc_pages_compact_quant(c, bits, table, lens, s["idx"], s["every"], *s["pool"], s["state"])
        table, lens = table[s["held"]:], lens[s["held"]:]
    elif kind != "read":
        kvc.kvc_pages_truncate(c, table, lens, s["base"], s["state"])   # what the pass before added goes back
        kvc.kvc_pages_append_quant(c, bits, table, lens, s["count"], s["row"], s["step"], *s["new"], *s["pool"], s["state"])
    kvc.kvc_pages_read_quant(c, bits, table, lens, s["from"], s["count"], s["to"], 1, *s["pool"], *s["out"], s["state"])
    return {"k": s["out"][0], "v": s["out"][1], "len": lens}


def _run_quant(s):
    if own:
        return _run_quant_own(s)
    c, kind = s["case"], s["case"]["kind"]
    who, at = _parts(s["count"])
    slot = s["start"][who] + s["from"][who] + at
    if kind == "evict":      # the copy's rows: the kept ones', moved as they are
        old, slot = s["start"][who] + s["idx"][who, at], s["start"][who] + s["base"][who] + at
        s["held_rows"] = [[_put(r, slot, r[old]) for r in room] for room in s["held_rows"]]
        s["len"].copy_(s["count"])
    elif kind != "read":
        src = s["row"][who] + at * s["step"]
        s["held_rows"] = [[_put(r, slot, p) for r, p in zip(room, _quantise(x[src], c["bits"]))]
                          for room, x in zip(s["held_rows"], s["new"])]
        s["len"].copy_(s["base"] + s["count"])
    k, v = (_put(o, s["to"][who] + at, _values(room[0][slot], room[1][slot], room[2][slot], c["dim"]).to(o.dtype))
            for o, room in zip(s["out"], s["held_rows"]))
    return {"k": k, "v": v, "len": s["len"]}


def _put(into, at, x):
    into[at] = x
    return into


def _exact_value(x, bits):
    """What x [rows][channels] stands for once it is held in so many bits, in 64 bits."""
    rows, d = x.shape
    y = torch.zeros((rows, _up(d, 32) * 32), dtype=torch.float64, device="cuda")
    y[:, :d] = x.double()
    y = y.reshape(rows, _up(d, 32), 32)
    low = torch.minimum(y.min(-1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
    high = torch.maximum(y.max(-1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
    n = 2 ** bits - 1
    t = ((high - low).float().double() / n).float().double()   # the format's own rounding
    fraction, exponent = torch.frexp(t)       # t = fraction 2^exponent, fraction in [0.5, 1)
    s = (torch.ceil(fraction * 16) / 16 if bits == 4 else torch.where(fraction > 0.5, 1.0, 0.5)) * 2.0 ** exponent.double()
    s = torch.where(t > 2.0 ** -126, s, 2.0 ** -126)
    factor = (1 / s).float().double()         # and this one
    z = torch.round((-low * factor).float().double())
    code = torch.round((y * factor[..., None]).float().double()) + z[..., None]
    code = torch.minimum(torch.maximum(code, torch.zeros_like(code)), torch.full_like(code, n))
    return ((code - z[..., None]) * s[..., None]).reshape(rows, -1)[:, :d]


def _exact_quant(c, seed):
    base, rows, held = _quant_sizes(c)
    g, d, dt, kind = _generator(seed), c["dim"], F[c["dtype"]], c["kind"]
    first = [_rows(g, sum(base), d, dt, strong) for strong in (True, False)]
    count, lens = (torch.tensor(x, device="cuda", dtype=torch.int32) for x in (rows, base))
    who, at = _parts(count)
    to = _starts(count)[who] + at
    if kind in ("token", "prompt"):
        x = [_rows(g, sum(rows), d, dt, strong) for strong in (True, False)]
        h = c["heads"]
        src = (_starts(count[::h])[who // h] + at) * h + who % h if kind == "token" else to
        left = lens + count
    elif kind == "read":
        x, left = first, lens
        src = _starts(lens)[who] + ((lens - count) // 2)[who] + at
    else:
        x, left = first, count
        span = (lens / count.clamp(min=1)).double()[:, None]
        k = max(1, max(rows))
        place = ((torch.arange(k, device="cuda") + torch.rand((held, k), generator=g, device="cuda", dtype=torch.float64)) * span).long()
        src = _starts(lens)[who] + torch.minimum(place, (lens.long() - 1).clamp(min=0)[:, None])[who, at]
    out = []
    for y in x:
        o = torch.zeros((max(1, sum(rows)), d), dtype=torch.float64, device="cuda")
        for i in range(0, who.numel(), 1 << 18):
            o[to[i:i + (1 << 18)]] = _exact_value(y[src[i:i + (1 << 18)]], c["bits"])
        out.append(o)
    return {"k": out[0], "v": out[1], "len": None} if sum(rows) else {"k": None, "v": None, "len": None}


# ------------------------------------------------------------------ attention

def _attend_sizes(c):
    n = _spread(c["seqs"], c["n_lo"], c["n_hi"])
    lens = [x + n[i // c["kv_heads"]] for i, x in enumerate(_spread(c["seqs"] * c["kv_heads"], c["len_lo"], c["len_hi"]))]
    return n, lens


def _prepare_attend(c, g):
    n, lens = _attend_sizes(c)
    d, h, dt = c["dim"], c["kv_heads"], F[c["dtype"]]
    i32 = dict(device="cuda", dtype=torch.int32)
    s = dict(case=c, max_new=max(n), len=torch.tensor(lens, **i32))
    s["q_start"] = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), **i32)
    rows = [_rows(g, sum(lens), d, dt, strong) for strong in (True, False)]
    s["q"] = torch.randn((sum(n), c["q_heads"], d), generator=g, device="cuda").to(dt)
    if own:
        from eviction_kvc_score_gb300 import kvc
        ps, lists = c["page"], c["seqs"] * h
        pages = [_up(x, ps) for x in lens]
        n_pages = sum(pages) + 5
        s["cache"] = kvc.cache(n_pages, ps, d, max(pages) + 1, c["dtype"])
        state = torch.empty(kvc.kvc_pages_size(s["cache"], lists), device="cuda", dtype=torch.uint8)
        kvc.kvc_pages_init(s["cache"], state)
        size = kvc.kvc_quant_page_size(s["cache"], c["bits"])
        pool = [torch.zeros((n_pages, size), device="cuda", dtype=torch.uint8) for _ in range(2)]
        s["table"] = torch.full((lists, s["cache"].max_pages), -1, **i32)
        lens_now = torch.zeros_like(s["len"])
        kvc.kvc_pages_append_quant(s["cache"], c["bits"], s["table"], lens_now, s["len"], _starts(s["len"]), 1, *rows, *pool, state)
        # pages in no order, as after a while of serving
        place = torch.randperm(n_pages, generator=g, device="cuda")
        s["pool"] = [_put(torch.empty_like(p), place, p) for p in pool]
        s["table"] = torch.where(s["table"] >= 0, place[s["table"].clamp(min=0).long()].int(), s["table"])
        s["ws"] = torch.empty(kvc.kvc_attend_quant_workspace_size(s["cache"], c["bits"], c["q_heads"], h, c["seqs"], s["max_new"]),
                              device="cuda", dtype=torch.uint8)
        kvc.kvc_workspace_init(s["ws"])
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    else:
        s["rows"] = [_quantise(x[:sum(lens)], c["bits"]) for x in rows]
        # row of every place of a table of whole lists
        t = max(lens)
        s["row"] = (_starts(s["len"])[:, None] + torch.arange(t, device="cuda")).clamp(max=max(0, sum(lens) - 1)).view(c["seqs"], h, t)
    return s


def _run_attend(s):
    c = s["case"]
    if own:
        from eviction_kvc_score_gb300 import kvc
        kvc.kvc_attend_quant(s["cache"], c["bits"], s["q"], s["q_start"], s["table"], s["len"], *s["pool"], s["max_new"], s["out"],
                             s["ws"], lse=s["lse"])
        return [s["out"], s["lse"]]
    b, h, d = c["seqs"], c["kv_heads"], c["dim"]
    g, m = c["q_heads"] // h, s["max_new"]
    row = s["row"]
    t = row.shape[-1]
    n = s["q_start"][1:] - s["q_start"][:-1]
    token, key = torch.arange(m, device="cuda"), torch.arange(t, device="cuda")
    at = (s["q_start"][:-1, None] + token).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"].float()[at].view(b, m, h, g, d).permute(0, 2, 3, 1, 4).reshape(b, h, g * m, d)
    k, v = s["rows"]
    score = q @ _values(k[0][row], k[1][row], k[2][row], d).transpose(-1, -2)
    score.mul_(1 / math.sqrt(d))
    # token i of n sees the first len - n + i + 1 keys of its list
    sees = (s["len"].view(b, h, 1) - n[:, None, None] + token + 1)[:, :, None, :, None] > key
    score = score.view(b, h, g, m, t).masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, h, g * m, t) @ _values(v[0][row], v[1][row], v[2][row], d)).view(b, h, g, m, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    real = (token < n[:, None])
    o = o.permute(0, 3, 1, 2, 4)[real].reshape(s["q"].shape).to(s["q"].dtype)
    return [o, lse.permute(0, 3, 1, 2, 4)[real].reshape(s["q"].shape[:2]).contiguous()]


def _exact_attend(c, seed):
    n, lens = _attend_sizes(c)
    gen, d, h, dt = _generator(seed), c["dim"], c["kv_heads"], F[c["dtype"]]
    rows = [_rows(gen, sum(lens), d, dt, strong) for strong in (True, False)]
    q = torch.randn((sum(n), c["q_heads"], d), generator=gen, device="cuda").to(dt)
    g = c["q_heads"] // h
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    first = row = 0
    for i in range(c["seqs"]):
        for j in range(h):
            size = lens[i * h + j]
            k, v = (_exact_value(x[row:row + size], c["bits"]) for x in rows)
            row += size
            for u in range(0, n[i], 1024):
                w = min(n[i], u + 1024)
                x = q[first + u:first + w, j * g:(j + 1) * g].double()
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
    make = {"quant": _prepare_quant, "attend": _prepare_attend}[case["op"]]
    return make(dict(case), _generator(seed))


def run(state):
    return {"quant": _run_quant, "attend": _run_attend}[state["case"]["op"]](state)


def exact(case, seed):
    return {"quant": _exact_quant, "attend": _exact_attend}[case["op"]](dict(case), seed)


def _held_bytes(c):
    """Bytes of one row of K or V as it is held: codes, and a step and a zero code per group."""
    return c["dim"] * c["bits"] // 8 + 2 * _up(c["dim"], 32)


def work(case):
    c, size = case, 4 if case["dtype"] == "f32" else 2
    if c["op"] == "quant":
        _, rows, held = _quant_sizes(c)
        moved, d = sum(rows), c["dim"]
        # the rows' values out; what they come from in; and, but for a mere reading, the held rows out
        came = _held_bytes(c) if c["kind"] in ("read", "evict") else d * size
        kept = 0 if c["kind"] == "read" else _held_bytes(c)
        return {"bytes": 2 * moved * (d * size + came + kept) + 4 * sum(_up(r, c["page"]) for r in rows) + 16 * held
                + (4 * moved if c["kind"] == "evict" else 0), "flops": 0}
    n, lens = _attend_sizes(c)
    h, g = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    pairs = sum(m * x - m * (m - 1) // 2 for x, m in ((x, n[i // h]) for i, x in enumerate(lens)))
    return {"bytes": 2 * sum(lens) * _held_bytes(c) + 2 * sum(n) * c["q_heads"] * c["dim"] * size + 4 * sum(n) * c["q_heads"]
            + 4 * sum(_up(x, c["page"]) for x in lens),
            "flops": 4 * pairs * g * c["dim"]}
