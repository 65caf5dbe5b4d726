"""Plain 64-bit forms of the operators around a verify round: rotary
positions, sampling, and the books of a page pool (definitions of
include/stv.h, in numpy and Python)."""
from __future__ import annotations

import numpy as np

PAGE = 256


# ---------------------------------------------------------------- rotary ---

def pair_axes(sections, half, interleaved):
    n = len(sections)
    if not interleaved:
        return np.repeat(np.arange(n), sections)
    out = np.zeros(half, np.int64)
    for a in range(1, n):
        out[a:n * sections[a]:n] = a
    return out


def rope(x, pos, rotary_dim, sections, theta, interleaved=False, inverse=False):
    """x float64 [rows][heads][head_dim], pos int [axes][rows]."""
    h = rotary_dim // 2
    axis = pair_axes(sections, h, interleaved)
    phi = pos[axis].T.astype(np.float64) * theta ** (-2.0 * np.arange(h) / rotary_dim)
    if inverse:
        phi = -phi
    c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
    y = x.copy()
    a, b = x[..., :h], x[..., h:2 * h]
    y[..., :h] = a * c - b * s
    y[..., h:2 * h] = b * c + a * s
    return y


# -------------------------------------------------------------- sampling ---

def sample(x, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (id, logprob, gap) -- gap: how near u comes to a border of the
    token drawn, or top_p to a border of its own, in units of the mass."""
    x = np.asarray(x, np.float64)
    # -x ascending, stable: larger first, among equals the lower index
    order = np.argsort(-x, kind="stable")
    order = order[np.isfinite(x[order])]
    if order.size == 0 or np.isnan(x).any() or np.isposinf(x).any():
        return -1, -np.inf, 1.0
    t, top_p, min_p, u = (np.float64(np.float32(v)) for v in (t, top_p, min_p, u))
    if t == 0:
        return int(order[0]), 0.0, 1.0
    gap = 1.0
    if top_k > 0:
        order = order[:top_k]
    w = np.exp((x[order] - x[order[0]]) / t)
    if top_p < 1:
        run = np.cumsum(w)
        need = top_p * run[-1]
        n = 1 + int(np.sum(run < need))
        gap = float(np.min(np.abs(run - need)) / run[-1])
        w = w[:n]
    w = w[:max(1, int(np.sum(w >= min_p)))]
    run = np.cumsum(w)
    at = min(int(np.sum(run <= u * run[-1])), w.size - 1)
    before = run[at] - w[at]
    gap = min(gap, float(min(run[at] - u * run[-1], u * run[-1] - before if at else 1.0) / run[-1]))
    return int(order[at]), float(np.log(w[at] / run[-1])), gap


# ----------------------------------------------------------------- pages ---

class Books:
    """A page pool and what its pages hold (one array entry per page)."""

    def __init__(self, n_pages, max_seqs, stride):
        self.refs = np.zeros(n_pages, np.int32)
        self.tables = np.full((max_seqs, stride), -1, np.int32)
        self.counts = np.zeros(max_seqs, np.int32)
        self.ctx = np.zeros(max_seqs, np.int32)
        self.data = np.arange(1, n_pages + 1, dtype=np.int64)

    def free_pages(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def take(self, s):
        page = self.free_pages()[0]
        self.refs[page] = 1
        self.tables[s, self.counts[s]] = page
        self.counts[s] += 1
        return page

    def reserve(self, seqs, extra):
        for s in seqs:
            while self.counts[s] * PAGE < self.ctx[s] + extra:
                self.take(s)

    def fork(self, src, dst):
        # new pages come from what was free before the call
        for a, b in zip(src, dst):
            c = int(self.ctx[a])
            for e in range(c // PAGE):
                page = self.tables[a, e]
                self.refs[page] += 1
                self.tables[b, e] = page
            self.counts[b] = c // PAGE
            if c % PAGE:
                self.data[self.take(b)] = self.data[self.tables[a, c // PAGE]]
            self.ctx[b] = c

    def free(self, seqs):
        for s in seqs:
            for e in range(self.counts[s]):
                self.refs[self.tables[s, e]] -= 1
            self.tables[s, :self.counts[s]] = -1
            self.counts[s] = 0

    def compact(self):
        live = [i for i, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [i for i in range(n) if self.refs[i] == 0]
        where = np.full(self.refs.size, -1, np.int32)
        where[live] = live
        for a, b in zip([i for i in live if i >= n], holes):
            self.data[b] = self.data[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            where[a] = b
        for s in range(self.counts.size):
            for e in range(self.counts[s]):
                self.tables[s, e] = where[self.tables[s, e]]
        return where, n
