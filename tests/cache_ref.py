"""Plain definitions of the paged-cache operators, in 64 bits or exact, for
the tests: no code is shared with the library."""
import math

import torch


def attend(q, q_start, table, lens, k_pool, v_pool, scale):
    """(out, lse, reach, logit): fp64 attention of every token of q over its
    lists; reach = sum_r p_r |v_r|, logit = the largest sum_d |q_d k_d| scale a
    row sees (what error bounds are made of).  Tokens outside every sequence
    keep NaN."""
    n_tok, hq, d = q.shape
    b = len(q_start) - 1
    h = table.shape[0] // b
    g = hq // h
    ps = k_pool.shape[1]
    out = torch.full((n_tok, hq, d), math.nan, dtype=torch.float64, device=q.device)
    reach, lse = out.clone(), out[..., 0].clone()
    logit = torch.zeros((n_tok, hq), dtype=torch.float64, device=q.device)
    for i in range(b):
        n = q_start[i + 1] - q_start[i]
        for j in range(h):
            size = lens[i * h + j]
            pages = table[i * h + j, :-(-size // ps)].long()
            k = k_pool[pages].reshape(-1, d)[:size].double()
            v = v_pool[pages].reshape(-1, d)[:size].double()
            for t in range(n):
                sees = max(0, size - n + t + 1)
                at, hs = q_start[i] + t, slice(j * g, (j + 1) * g)
                if sees == 0:
                    out[at, hs], reach[at, hs], lse[at, hs] = 0, 0, -math.inf
                    continue
                x = q[at, hs].double()
                z = x @ k[:sees].T * scale
                p = torch.softmax(z, -1)
                out[at, hs] = p @ v[:sees]
                reach[at, hs] = p @ v[:sees].abs()
                lse[at, hs] = torch.logsumexp(z, -1)
                logit[at, hs] = (x.abs() @ k[:sees].abs().T).amax(-1) * abs(scale)
    return out, lse, reach, logit


def rope_frequencies(rot, theta, factor=1.0, alpha=1.0, beta=4.0, context=8192.0):
    f = []
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        turns = context * w / (2 * math.pi)
        g = 1.0 if factor <= 1 or turns >= beta else 0.0 if turns <= alpha else (turns - alpha) / (beta - alpha)
        f.append(w * (g + (1 - g) / factor))
    return torch.tensor(f, dtype=torch.float64)


def rope(x, pos, freq, interleaved, inverse=False, amplitude=1.0):
    """fp64 rotation of x [tokens][heads][D]."""
    y = x.double().clone()
    rot = 2 * freq.numel()
    ang = pos.double()[:, None, None] * freq.to(x.device)
    c, s = amplitude * torch.cos(ang), amplitude * torch.sin(ang) * (-1 if inverse else 1)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    u, w = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - w * s, u * s + w * c
    return y


class Pages:
    """A page pool as lists of rows: what every call has to leave behind."""

    def __init__(self, n_pages, page_rows, max_pages, n_lists):
        self.ps, self.max_pages = page_rows, max_pages
        self.holders = [0] * n_pages
        self.rows = {}                      # (page, row) -> whatever stands for the row
        self.table = [[] for _ in range(n_lists)]
        self.len = [0] * n_lists

    def free(self):
        return [p for p, n in enumerate(self.holders) if n == 0]

    def take(self, need):
        free = self.free()
        if sum(need) > len(free):
            return None
        got, at = [], 0
        for n in need:
            got.append(free[at:at + n])
            at += n
        for p in free[:at]:
            self.holders[p] = 1
        return got

    def pages(self, n):
        return -(-n // self.ps)

    def append(self, rows):
        """rows[i]: the new rows of list i.  False if nothing was done."""
        need, shared = [], []
        for i, new in enumerate(rows):
            n = len(new)
            if self.len[i] + n > self.max_pages * self.ps:
                return False
            cow = n > 0 and self.len[i] % self.ps > 0 and self.holders[self.table[i][self.len[i] // self.ps]] > 1
            shared.append(cow)
            need.append(self.pages(self.len[i] + n) - self.pages(self.len[i]) + cow if n else 0)
        got = self.take(need)
        if got is None:
            return False
        for i, new in enumerate(rows):
            pages = got[i]
            if shared[i]:
                old, own = self.table[i][-1], pages.pop(0)
                self.holders[old] -= 1
                for r in range(self.len[i] % self.ps):
                    self.rows[own, r] = self.rows[old, r]
                self.table[i][-1] = own
            self.table[i] = self.table[i] + pages
            for r in new:
                self.rows[self.table[i][self.len[i] // self.ps], self.len[i] % self.ps] = r
                self.len[i] += 1
        return True

    def fork(self, src):
        for i, s in enumerate(src):
            if s >= 0 and s < len(src) and self.len[i] == 0 and src[s] < 0:
                self.table[i], self.len[i] = list(self.table[s]), self.len[s]
                for p in self.table[i]:
                    self.holders[p] += 1

    def list_rows(self, i):
        return [self.rows[self.table[i][r // self.ps], r % self.ps] for r in range(self.len[i])]

    def compact(self, idx):
        """idx[i]: kept rows of list i, or None."""
        got = self.take([0 if x is None else self.pages(len(x)) for x in idx])
        if got is None:
            return False
        for i, x in enumerate(idx):
            if x is None:
                continue
            rows = self.list_rows(i)
            for r, j in enumerate(x):
                self.rows[got[i][r // self.ps], r % self.ps] = rows[j]
            for p in self.table[i]:
                self.holders[p] -= 1
            self.table[i], self.len[i] = got[i], len(x)
        return True

    def truncate(self, new):
        for i, n in enumerate(new):
            if 0 <= n < self.len[i]:
                for p in self.table[i][self.pages(n):]:
                    self.holders[p] -= 1
                self.table[i], self.len[i] = self.table[i][:self.pages(n)], n
