"""Plain 64-bit forms of the drafter's side of a round (definitions of
include/stv.h): ragged pages and rows, the 16-bit paged cache, attention over
it, and acceptance by probabilities."""
from __future__ import annotations

import numpy as np
import torch

import speculative_tree_verify_bit_gb300 as stv

PAGE = 256


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), device="cuda").to(dtype)


# ------------------------------------------------------------- a cache ------

class Drafter:
    """A pool with sequences of given lengths on shuffled pages; every element
    that belongs to no key holds `fill`."""

    def __init__(self, lens, hkv, hd, dtype, seed=0, spare=2, fill=float("nan"), max_seqs=None, n_pages=None):
        rng, g = np.random.default_rng(seed), torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        held = [-(-n // PAGE) for n in lens]
        n_pages = n_pages or sum(held) + spare
        max_seqs = max_seqs or max(1, len(lens))
        self.hkv, self.hd, self.dtype, self.lens = hkv, hd, dtype, list(lens)
        self.data = torch.full((n_pages, hkv, 2, PAGE, hd), fill, dtype=dtype, device="cuda")
        tables = np.full((max_seqs, max(held + [1]) + 1), -1, np.int32)
        perm, at = rng.permutation(n_pages), 0
        for s, n in enumerate(lens):
            tables[s, :held[s]] = perm[at:at + held[s]]
            at += held[s]
            for e in range(held[s]):
                k = min(PAGE, n - e * PAGE)
                self.data[int(tables[s, e]), :, :, :k] = torch.randn((hkv, 2, k, hd), generator=g, device="cuda").to(dtype)
        refs = np.zeros(n_pages, np.int32)
        refs[perm[:at]] = 1
        self.pool = stv.PagePool(dev(refs), dev(tables), dev(held + [0] * (max_seqs - len(lens))))
        self.layer = stv.RowCache(self.data)
        self.g = g

    def rows(self, n, heads):
        return torch.randn((n, heads, self.hd), generator=self.g, device="cuda").to(self.dtype)

    def keys(self, s, end):
        """K and V of sequence s's first `end` tokens, fp64 [end][hkv][2][hd]."""
        if end == 0:
            return torch.zeros((0, self.hkv, 2, self.hd), dtype=torch.float64, device="cuda")
        pages = self.pool.tables[s, :-(-end // PAGE)].long()
        return self.data[pages].permute(0, 3, 1, 2, 4).reshape(-1, self.hkv, 2, self.hd)[:end].double()


def visible(pos, end, window, sinks, causal, device="cuda"):
    """[len(pos)][end]: whether the row at pos sees the key."""
    k = torch.arange(end, device=device)[None]
    p = torch.as_tensor(pos, device=device)[:, None]
    see = (k <= p) if causal else torch.ones_like(k <= p)
    if window:
        see = see & ((k > p - window) | (k < sinks))
    return see


def attention(d, q, entries, window=0, sinks=0, causal=True, scale=None, hidden=()):
    """entries: (sequence, ctx, first row, rows).  Returns o and the
    elementwise bound of what the kernels may be off by (fp64, 0 for rows
    outside the entries).  hidden: keys of any sequence that have no page."""
    hq, hd = q.shape[1], q.shape[2]
    g, scale = hq // d.hkv, hd ** -0.5 if scale is None else scale
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    # a rounding is off by at most half a step
    half = torch.finfo(d.dtype).eps / 2
    for s, ctx, row, n in entries:
        if n == 0:
            continue
        end = ctx + n
        kv = d.keys(s, end)
        see = visible(np.arange(ctx, end), end, window, sinks, causal)
        for k0 in hidden:
            see[:, k0:k0 + PAGE] = False
        used = see.any(0)
        kv, see = kv[used], see[:, used]
        for h in range(hq):
            qq = q[row:row + n, h].double()
            kk, vv = kv[:, h // g, 0], kv[:, h // g, 1]
            x = (qq @ kk.T * scale).masked_fill(~see, -float("inf"))
            w = torch.softmax(x, 1).nan_to_num(0.0)  # a row that sees nothing is zero
            o[row:row + n, h] = w @ vv
            # fp32 sums of hd products, the scaled score and 2^x: relative to 1
            size = (qq.abs() @ kk.abs().T * scale).masked_fill(~see, 0).amax(1, keepdim=True) if kk.shape[0] else 0
            delta = size * (hd + 8) * 2.0 ** -24 + 2.0 ** -21
            spread = w @ vv.abs()
            # P rounded (in the sum too), fp32 sums over the keys, the result rounded; fp16 P below
            # 2^-14 of a row's largest is off by 2^-25
            tol[row:row + n, h] = (half * o[row:row + n, h].abs() + spread * (2 * half + 2 * delta + kk.shape[0] * 2.0 ** -23)
                                   + (kk.shape[0] * 2.0 ** -25 * vv.abs().max() if kk.shape[0] and d.dtype == torch.float16
                                      else 0) + 1e-30)
    return o, tol


# ---------------------------------------------------------- acceptance ------

def accept(parent, ids, p, q, u, distinct):
    """One sequence; p, q float64 [T][vocab] (q None: certain drafts), u of the
    tests and of the draw.  Returns (nodes of the path, out_ids, gap): gap, how near a decision
    comes to its border, relative to 1."""
    t, vocab = p.shape
    at, path, out, gap = 0, [0], [], 1.0
    while True:
        r, z = p[at].copy(), 1.0
        s = None if q is None else q[at].copy()
        down = None
        for c in [i for i in range(at + 1, t) if parent[i] == at]:
            x = ids[c]
            if not 0 <= x < vocab:
                continue
            share = 1.0 if s is None else s[x]
            gap = min(gap, abs(u[c] * share * z - r[x]) or 1.0)  # equal to the last bit: no rounding decides
            if u[c] * share * z < r[x]:
                down = c
                break
            left = r.copy()
            if s is None:
                left[x] = 0
            else:
                left = np.maximum(r - z * s, 0)
            if left.sum() > 0:
                r, z = left, left.sum()
            if s is not None and distinct:
                s[x] = 0
                s = s / s.sum() if s.sum() > 0 else s
        if down is None:
            break
        out.append(int(ids[down]))
        path.append(down)
        at = down
    run = np.cumsum(r)
    gap = min(gap, float(np.min(np.abs(run - u[0] * run[-1])) / run[-1]) or 1.0)
    out.append(int(np.nonzero(run > u[0] * run[-1])[0][0]))
    return path, out, gap
