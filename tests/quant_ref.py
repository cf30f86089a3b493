"""Plain definitions of rows held in 4 or 8 bits and of attention over them, in
64 bits, for the tests: no code is shared with the library."""
import math

import torch

N = {4: 15, 8: 255}


def fl(x):
    """Rounded to fp32."""
    return x.float().double()


def pow2(e):
    """2^e, exactly, for whole e (a GPU's power function is not exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantise(x, bits):
    """Codes n, steps s and zero codes z of the groups of x [rows][D]: fp64
    [rows][D] (each channel with its group's step and zero code); s is NaN where
    the group stands for NaN."""
    rows, d = x.shape
    parts = []
    for at in range(0, d, 32):
        y = x[:, at:at + 32].double()
        lo = torch.clamp(y.nan_to_num(0, 0, 0).amin(1), max=0)
        hi = torch.clamp(y.nan_to_num(0, 0, 0).amax(1), min=0)
        bad = ~(y.abs() < 2.0 ** 126).all(1)
        y = torch.where(bad[:, None], 0.0, y)
        lo, hi = torch.where(bad, 0.0, lo), torch.where(bad, 0.0, hi)
        t = fl(fl(hi / 2 - lo / 2) / (N[bits] / 2))
        e = torch.floor(torch.log2(torch.clamp(t, min=2.0 ** -126)))
        e = torch.where(pow2(e) > t, e - 1, e)          # log2 may round up
        unit = pow2(e - 3) if bits == 4 else pow2(e)
        s = torch.ceil(t / unit) * unit
        if bits == 8:
            s = torch.where(s > pow2(e), pow2(e + 1), s)
        s = torch.clamp(s, min=2.0 ** -126)
        inv = fl(1 / s)
        z = torch.round(fl(-lo * inv))
        n = torch.clamp(torch.round(fl(y * inv[:, None])) + z[:, None], 0, N[bits])
        s = torch.where(bad, math.nan, s)
        w = y.shape[1]
        parts.append((n, s[:, None].expand(-1, w), z[:, None].expand(-1, w)))
    return tuple(torch.cat([p[i] for p in parts], 1) for i in range(3))


def stands(x, bits):
    n, s, z = quantise(x, bits)
    return (n - z) * s


def wide(x, bits):
    """(n + z) s: what the sums over codes are made of, and errors are bounded by."""
    n, s, z = quantise(x, bits)
    return (n + z) * s


def attend(q, starts, k, v, scale, bits):
    """fp64 attention of q [tokens][H_q][D] over lists of rows k[i], v[i], the
    rows as they are before they are quantised.  A dict: out, lse; reach = sum p |v|,
    reach_w the same of wide(); logit_w = the largest sum_d |q_d| wide(k)_d scale a
    row sees, logit_top the same with the token's largest |q|; step = the largest
    step of V.  NaN where no sequence has the token."""
    n_tok, hq, d = q.shape
    b = len(starts) - 1
    h = len(k) // b
    g = hq // h
    r = {x: torch.full((n_tok, hq, d), math.nan, dtype=torch.float64, device=q.device) for x in ("out", "reach", "reach_w")}
    r.update({x: torch.full((n_tok, hq), math.nan, dtype=torch.float64, device=q.device) for x in ("lse", "logit_w", "logit_top", "step")})
    for i in range(b):
        n = starts[i + 1] - starts[i]
        for j in range(h):
            kk, vv = k[i * h + j], v[i * h + j]
            size = kk.shape[0]
            ks, kw, vs, vw = stands(kk, bits), wide(kk, bits), stands(vv, bits), wide(vv, bits)
            step = quantise(vv, bits)[1].nan_to_num(0)
            for t in range(n):
                sees = max(0, size - n + t + 1)
                at, hs = starts[i] + t, slice(j * g, (j + 1) * g)
                if sees == 0:
                    for x in r:
                        r[x][at, hs] = -math.inf if x == "lse" else 0
                    continue
                x = q[at, hs].double()
                z = x @ ks[:sees].T * scale
                p = torch.softmax(z, -1)
                r["out"][at, hs] = p @ vs[:sees]
                r["reach"][at, hs] = p @ vs[:sees].abs()
                r["reach_w"][at, hs] = p @ vw[:sees]
                r["lse"][at, hs] = torch.logsumexp(z, -1)
                r["logit_w"][at, hs] = (x.abs() @ kw[:sees].T).amax(-1) * abs(scale)
                r["logit_top"][at, hs] = x.abs().amax(-1) * kw[:sees].sum(-1).amax() * abs(scale)
                r["step"][at, hs] = step.max()
    return r


def near(out, want, logit=4):
    """None if an output is as near to the fp64 definition as it has to be, else how far off it is; `logit`: the
    size of the logits that decide it.

    fp32: 2e-6 of the norm.  T additions that round leave u sqrt(T / 6) of it (4,000 rows: 1.5e-6), and
    tiles are added up apart from each other.  P or Q in two bf16 pieces, cut off, would lose 2^-17 of every
    weight on average, 7.6e-6.  A weight errs by its logit's error: sums and products of fp32 leave 2^-24 of that
    each, a tensor core's sum 2^-23; four of the latter are taken for logits above 4 (below they are in the 2e-6).
    bf16: where `out` is the definition's value plus an error of 2^-15 of its root mean square s and is then rounded
    to a step of 0.72 2^-8 |out| on average, one value in E |error| / step is not the nearest: the mean of s / |out|
    over a normal distribution, cut off where the step is the error, is 0.8 ln 128, together 3.3%; 4% may be.
    Probabilities of 16 bits err by 2^-18 / sqrt(3), those of 11 bits by 2^-12 / sqrt(3): 9%."""
    real = want.isfinite()
    assert out[real].isfinite().all()
    x, y = out[real], want[real]
    if out.dtype == torch.float32:
        off = ((x.double() - y).norm() / y.norm()).item()
        return None if off <= 2e-6 + 4 * max(0, logit - 4) * 2.0 ** -23 else off
    other = (x != y.to(out.dtype)).double().mean().item()
    return None if other <= 0.04 else other
