"""stv_tree_accept_probs where a decision lies close to its border: answers
from exact rational numbers, inputs searched so that single precision, or a
product that was not rounded where it should have been, decides otherwise."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from drafterkit import dev

pytestmark = pytest.mark.gpu


def call(parent, ids, p, q, u, distinct=False):
    n, t = np.shape(parent)
    out = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((n,), (n, t), (n, t))]
    status = dev([0])
    f32 = lambda x: None if x is None else torch.as_tensor(np.ascontiguousarray(x, np.float32), device="cuda")
    stv.stv_tree_accept_probs(dev(parent), dev(ids), f32(p), f32(q), f32(u), *out, distinct=distinct, dev_status=status)
    assert status.item() == 0
    return [o.cpu().numpy() for o in out]


def units(row):
    """fp32 values as whole numbers of 2^-149."""
    return np.array([int(Fraction(float(x)) * (1 << 149)) for x in row], dtype=object)


def exact(parent, ids, p, q, u, distinct):
    """The definition in whole numbers: R = r / d, Z = z / d, S = s / m; p, q fp32 [T][vocab].
    Returns (path, out_ids, gap): gap, how near a decision after a rejection, or the last token's,
    comes to its border, relative to the two sides."""
    at, path, out, gap = 0, [0], [], 1.0
    near = lambda a, b: float(Fraction(abs(a - b), max(a, b))) if a != b else 1.0
    uu = units(u)
    one = 1 << 149
    while True:
        r, d, z = units(p[at]), one, one
        s, m = (None, 1) if q is None else (units(q[at]), one)
        first, down = True, None
        for c in [i for i in range(at + 1, len(parent)) if parent[i] == at]:
            x = int(ids[c])
            share = 1 if s is None else s[x]
            a, b = uu[c] * z * share, r[x] * m * one
            if not first:
                gap = min(gap, near(a, b))
            if a < b:
                down = c
                break
            first = False
            if s is None:
                left, scale = r.copy(), 1
                left[x] = 0
            else:
                left, scale = np.maximum(r * m - z * s, 0), m
            if left.any():
                r, d, z = left, d * scale, left.sum()
            if s is not None and distinct:
                s[x] = 0
                m = int(s.sum()) or m
        if down is None:
            break
        out.append(int(ids[down]))
        path.append(down)
        at = down
    run = np.cumsum(r)
    past = run * one > uu[0] * run[-1]
    x = int(np.nonzero(past)[0][0])
    for k in (x - 1, x):
        if k >= 0 and run[k]:
            gap = min(gap, float(Fraction(abs(run[k] * one - uu[0] * run[-1]), run[-1] * one)) or 1.0)
    return path, out + [x], gap


def check(parent, ids, p, q, u, distinct, nearest=0.0, furthest=1.0):
    """All sequences against `exact`; their decisions lie between the two gaps."""
    n, t = parent.shape
    got = call(parent, ids, p, q, u, distinct)
    wrong = []
    for s in range(n):
        rs = slice(s * t, (s + 1) * t)
        path, out, gap = exact(parent[s], ids[s], p[rs], None if q is None else q[rs], u[s], distinct)
        assert nearest < gap < furthest, gap
        m = len(path)
        if (got[0][s], got[1][s, :m].tolist(), got[2][s, :m].tolist()) != (m, path, out):
            wrong.append((s, gap, path, out, [g[s].tolist() for g in got]))
        assert (got[2][s] != -9).all() and (got[1][s] != -9).all()
    assert not wrong, (len(wrong), wrong[:3])


def test_first_children_are_decided_exactly(gpu):
    """u q against the numbers of 24 bits on either side of it: the low half of the product decides."""
    rng = np.random.default_rng(1)
    n, vocab = 3000, 8
    u = np.float32(rng.random(n) * 0.999 + 0.0005)
    share = np.float32(2.0 ** -rng.uniform(0, 40, n))
    prod = u.astype(np.float64) * share.astype(np.float64)  # 48 bits: exact
    near = np.float32(prod)
    p_x = np.where(rng.random(n) < 0.5, near, np.where(near > prod, np.nextafter(near, np.float32(0)),
                                                       np.nextafter(near, np.float32(1)))).astype(np.float32)
    p, q = np.zeros((2 * n, vocab), np.float32), np.full((2 * n, vocab), 0.1, np.float32)
    p[:, 0] = 0.5
    p[::2, 3], q[::2, 3] = p_x, share
    parent, ids = np.tile([-1, 0], (n, 1)), np.tile([0, 3], (n, 1))
    uu = np.stack([np.full(n, 0.25, np.float32), u], 1)
    nc, path, out = call(parent, ids, p, q, uu)
    want = np.array([Fraction(float(a)) * Fraction(float(b)) < Fraction(float(c)) for a, b, c in zip(u, share, p_x)])
    assert 0.3 < want.mean() < 0.7
    assert (nc == 1 + want).all(), np.nonzero(nc != 1 + want)[0][:10]


def near_border(rng, ratio_of, tries=1 << 16):
    """A p(x) and a u, of 24 bits both, such that u is next to the border ratio_of(p(x)), on either side: the
    nearest of `tries` neighbouring p(x), but no nearer than 2^-44 F / Z: R = p - F q is off by up to 2^-45 F q,
    and u - R / (Z S) so by 2^-45 F / Z (ratio_of by some 2^-50).  ratio_of: R / (Z S), and F / Z."""
    coarse = np.arange(1, 4097) * 2.0 ** -14
    r, _ = ratio_of(coarse)
    start = rng.choice(coarse[(r > 0.1) & (r < 0.9)])
    x = (np.float32(start) + np.arange(tries) * 2.0 ** -28).astype(np.float32).astype(np.float64)
    r, far = ratio_of(x)
    u = np.clip(r, 0, 0.99).astype(np.float32).astype(np.float64)
    side = u < r if rng.random() < 0.5 else u > r
    off = np.where(side & (np.abs(u - r) > 2.0 ** -44 * far), np.abs(u - r), 1.0)
    k = int(np.argmin(off))
    assert off[k] < 2.0 ** -35
    return np.float32(x[k]), np.float32(u[k])


@pytest.mark.parametrize("distinct", [False, True])
@pytest.mark.parametrize("before", [1, 2, 5])
def test_later_children_close_to_the_border(gpu, before, distinct):
    """The last of `before` + 1 children, after rejections of tokens that the target does not have:
    u Z S and R = p - F q as near to one another as the documented error allows."""
    rng = np.random.default_rng(10 * before + distinct)
    n, t, vocab = 40, before + 2, 24
    p, q = np.zeros((n * t, vocab), np.float32), np.zeros((n * t, vocab), np.float32)
    ids, u = np.zeros((n, t), np.int64), np.zeros((n, t), np.float32)
    for s in range(n):
        pr, qr = rng.random(vocab), rng.random(vocab)
        gone = rng.choice(vocab - 1, before, replace=False) + 1  # the rejected tokens; x = 0
        qr[gone] = 0.02 + 0.3 * rng.random(before)
        pr[gone] = 0
        qr[0] = 0.1 + 0.1 * rng.random()
        pr, qr = np.float32(pr / pr.sum() * 0.8).astype(np.float64), np.float32(qr / qr.sum()).astype(np.float64)
        others = np.setdiff1d(np.arange(1, vocab), gone)

        def ratio(x):
            r, z, w, m, f = x.copy(), np.ones_like(x), qr.copy(), 1.0, np.zeros_like(x)
            rest = np.tile(pr[others][:, None], (1, len(x)))
            for y in gone:
                r = r - z * w[0] / m
                f += z / m
                rest = np.maximum(rest - z * w[others][:, None] / m, 0)
                z = np.maximum(r, 0) + rest.sum(0)
                if distinct:
                    w[y] = 0
                    m = w.sum()
            return r / (z * (w[0] / m)), f / z

        pr[0], u[s, t - 1] = near_border(rng, ratio)
        p[s * t], q[s * t] = pr, qr
        p[s * t + 1:(s + 1) * t, 1] = 1
        q[s * t + 1:(s + 1) * t, 1] = 1
        ids[s, 1:] = list(gone) + [0]
        u[s, :-1] = np.float32(rng.uniform(0.2, 0.8, t - 1))
    check(np.tile([-1] + [0] * (t - 1), (n, 1)), ids, p, q, u, distinct, furthest=2.0 ** -30)


@pytest.mark.parametrize("drafts", ["replaced", "distinct", "certain"])
@pytest.mark.parametrize("vocab,n", [(600, 24), (4097, 12), (70001, 3)])
def test_last_tokens_close_to_the_border(gpu, vocab, n, drafts):
    """u[0] times the mass next to a running sum, after rejections; every fourth sequence at the border of a
    quarter, of a warp's and of a thread's share of the row."""
    rng = np.random.default_rng(vocab)
    t = 4
    p, q = (np.exp(1.5 * rng.normal(size=(n * t, vocab))) for _ in range(2))
    ids, u = np.zeros((n, t), np.int64), np.float32(rng.uniform(0.3, 0.9, (n, t)))
    for s in range(n):
        ids[s, 1:] = rng.choice(vocab, t - 1, replace=False)
        p[s * t, ids[s, 1:]] = 0 if drafts != "certain" else p[s * t].sum() * 0.01
        q[s * t, ids[s, 1:]] = q[s * t].sum() * np.array([0.1, 0.05, 0.2])
    p, q = (np.float32(x / x.sum(1, keepdims=True)) for x in (p, q))
    for s in range(n):
        r, z, w = p[s * t].astype(np.float64), 1.0, q[s * t].astype(np.float64)
        for c in ids[s, 1:]:
            if drafts == "certain":
                r[c] = 0
            else:
                r = np.maximum(r - z * w, 0)
            z = r.sum()
            if drafts == "distinct":
                w[c] = 0
                w /= w.sum()
        edge = np.cumsum(r) / r.sum()
        near = edge.astype(np.float32)
        off = np.abs(near - edge)
        ok = np.nonzero((off > 2.0 ** -40) & (edge < 0.999) & (r > 0))[0]
        if s % 4 == 3:
            ok = ok[np.argsort(np.abs(ok + 1 - vocab // 4 * (1 + s // 4 % 3)))[:1]]
        u[s, 0] = near[ok[int(np.argmin(off[ok]))]]
    check(np.tile([-1, 0, 0, 0], (n, 1)), ids, p, None if drafts == "certain" else q, u, drafts == "distinct",
          nearest=2.0 ** -41)


def test_first_children_of_tiny_shares(gpu):
    """u q where its low half, or all of it, lies below fp32's smallest number."""
    rng = np.random.default_rng(2)
    n, vocab = 3000, 4
    tiny = np.float32(2.0 ** -149)
    share = np.float32(2.0 ** -rng.uniform(80, 146, n))
    share[::7] = np.float32(tiny * rng.integers(1, 9, len(share[::7])))
    u = np.float32(rng.random(n) * 0.999 + 0.0005)
    prod = u.astype(np.float64) * share.astype(np.float64)
    near = np.float32(prod)
    other = np.where(near > prod, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(1)))
    p_x = np.where(rng.random(n) < 0.5, near, other).astype(np.float32)
    p, q = np.zeros((2 * n, vocab), np.float32), np.full((2 * n, vocab), 0.1, np.float32)
    p[:, 0] = 0.5
    p[::2, 3], q[::2, 3] = p_x, share
    uu = np.stack([np.full(n, 0.25, np.float32), u], 1)
    nc, path, out = call(np.tile([-1, 0], (n, 1)), np.tile([0, 3], (n, 1)), p, q, uu)
    want = np.array([Fraction(float(a)) * Fraction(float(b)) < Fraction(float(c)) for a, b, c in zip(u, share, p_x)])
    assert 0.3 < want.mean() < 0.7
    assert (nc == 1 + want).all(), (int((nc != 1 + want).sum()), np.nonzero(nc != 1 + want)[0][:10])
