"""Plain references of the cache operators: rotary positions and attention in 64 bits, and the cache's
books as lists.  Written from the definitions in include/dspark.h; CPU only."""
import math

import torch

UNIT = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}  # unit roundoff


def rotary(x, positions, freqs, *, layout="half", amplitude=1.0, backward=False):
    """x [tokens, heads, dim] double; freqs: turns a position, floats [rotary_dim / 2]."""
    half = len(freqs)
    f = torch.tensor(freqs, dtype=torch.float64)
    angle = positions.double()[:, None] * f * (2.0 * math.pi)
    cos, sin = amplitude * torch.cos(angle)[:, None], amplitude * torch.sin(angle)[:, None]
    if backward:
        sin = -sin
    y = x.clone()
    at = torch.arange(half)
    i, j = (at, at + half) if layout == "half" else (2 * at, 2 * at + 1)
    a, b = x[..., i], x[..., j]
    y[..., i] = a * cos - b * sin
    y[..., j] = b * cos + a * sin
    return y


def row_tokens(pool, table, layer, row, length):
    """k, v [length, heads, dim] of a row, double, by walking its pages."""
    page_size = pool.shape[4]
    k = [pool[table[row, j // page_size], layer, 0, :, j % page_size] for j in range(length)]
    v = [pool[table[row, j // page_size], layer, 1, :, j % page_size] for j in range(length)]
    empty = torch.zeros((0, pool.shape[3], pool.shape[5]), dtype=torch.float64)
    return (torch.stack(k).double(), torch.stack(v).double()) if length else (empty, empty)


def attention(q, k, v, n, *, causal, window, scale):
    """One sequence: q [n, q_heads, dim], k, v [length, kv_heads, dim], all double.  Returns out, lse, sum_j w_j |v_j|
    (what weights' roundings are relative to), sum over seen keys of |v_j|, and the largest sum_e |q_e k_e| * scale."""
    length, group = k.shape[0], q.shape[1] // k.shape[1]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    weight_abs, plain_abs, dot_abs = torch.zeros_like(q), torch.zeros_like(q), 0.0
    j = torch.arange(length)
    for i in range(n):
        p = length - n + i
        seen = torch.ones(length, dtype=torch.bool)
        if causal:
            seen &= j <= p
        if window:
            seen &= j > p - window
        if not seen.any():
            continue
        for h in range(q.shape[1]):
            kk, vv = k[seen, h // group], v[seen, h // group]
            s = (kk @ q[i, h]) * scale
            dot_abs = max(dot_abs, float((kk.abs() @ q[i, h].abs()).max()) * scale)
            lse[i, h] = torch.logsumexp(s, 0)
            w = torch.exp(s - lse[i, h])
            out[i, h] = w @ vv
            weight_abs[i, h] = w @ vv.abs()
            plain_abs[i, h] = vv.abs().sum(0)
    return out, lse, weight_abs, plain_abs, dot_abs


class Books:
    """The cache's books by their definition: tables as lists, a page free when no row holds it."""

    def __init__(self, num_pages, max_pages, page_size, rows):
        self.num_pages, self.max_pages, self.page = num_pages, max_pages, page_size
        self.pages = {r: [] for r in range(rows)}
        self.length = {r: 0 for r in range(rows)}
        self.moves = []  # ((page, slot) from, (page, slot) to) of the last call, as of before it

    def refs(self):
        out = [0] * self.num_pages
        for pages in self.pages.values():
            for p in pages:
                out[p] += 1
        return out

    def _free(self):
        return iter([p for p, n in enumerate(self.refs()) if n == 0])

    def _need(self, tokens):
        return -(-tokens // self.page)

    def extend(self, rows, counts):
        free, was = self._free(), {r: list(p) for r, p in self.pages.items()}
        for r, c in zip(rows, counts):
            while len(self.pages[r]) < self._need(self.length[r] + c):
                page = next(free, None)
                if page is None or len(self.pages[r]) == self.max_pages:
                    self.pages = was
                    return False
                self.pages[r].append(page)
        for r, c in zip(rows, counts):
            self.length[r] += c
        return True

    def free(self, rows):
        for r in rows:
            self.pages[r], self.length[r] = [], 0

    def fork(self, src, dst):
        free, was, length = self._free(), {r: list(p) for r, p in self.pages.items()}, dict(self.length)
        self.moves, now = [], {}
        for s, d in zip(src, dst):
            if s == d:
                continue
            pages, tail = list(was[s]), length[s] % self.page
            if tail:
                page = next(free, None)
                if page is None:
                    return False
                self.moves += [((pages[-1], t), (page, t)) for t in range(tail)]
                pages[-1] = page
            now[d] = (pages, length[s])
        for d, (pages, n) in now.items():
            self.pages[d], self.length[d] = pages, n
        return True

    def compact(self, rows, start, kept):
        free, refs = self._free(), self.refs()
        self.moves, now = [], {}
        for r, st, keep in zip(rows, start, kept):
            tokens = list(range(st)) + list(keep)
            old = self.pages[r]
            pages = old[: self._need(len(tokens))]
            for j in range(st // self.page, len(pages)):
                if refs[pages[j]] > 1:
                    pages[j] = next(free, None)
                    if pages[j] is None:
                        return False
            for at in range(st // self.page * self.page, len(tokens)):
                t = tokens[at]
                self.moves.append(((old[t // self.page], t % self.page), (pages[at // self.page], at % self.page)))
            now[r] = (pages, len(tokens))
        for r, (pages, n) in now.items():
            self.pages[r], self.length[r] = pages, n
        return True

    def moved(self, pool):
        """The pool [pages, layers, 2, heads, slots, dim] after the last call's moves."""
        new = pool.clone()
        for (p, s), (to, t) in self.moves:
            new[to, :, :, :, t] = pool[p, :, :, :, s]
        return new

    def table(self):
        rows = len(self.pages)
        out = torch.full((rows, self.max_pages), -1, dtype=torch.int32)
        for r, pages in self.pages.items():
            out[r, : len(pages)] = torch.tensor(pages, dtype=torch.int32)
        return out
