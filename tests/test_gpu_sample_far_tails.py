"""stv_sample where much of a row lies far below its largest logit.

A weight is an integer of at least 2^44 for the largest, off by less than
2^-28 of itself and one unit, 2^-44 of the largest (a value cut to a whole
number whose last bit is then set).  Equal tokens are all off by the same, so
with n tokens and m their mass in units of the largest's, a share f = A / M of
the mass is off by at most
    (dA (M - A) + d(M - A) A) / M^2  <=  f (1 - f) 2^-27 + n 2^-44 / m
                                     <=  2^-29 + n 2^-44 / m,
at the cut of top_p and at the draw.  The token drawn must own, in the exact
order and masses, a stretch that u comes so near to, and top_p a cut.  logprob
is off by the fp32 rounding, 2^-24 of its value, the weight's and the mass's
2^-28 and the logarithms (2^-27 in all), and n 2^-44 / m."""
import numpy as np
import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def draw(logits, u, t, k, p):
    n = logits.shape[0]
    ids = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((n,), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = lambda v, dt: torch.tensor([v], dtype=dt, device="cuda")
    stv.stv_sample(logits, u, ids, lp, f(t, torch.float32), f(k, torch.int32), f(p, torch.float32), None, n,
                   dev_status=status)
    assert int(status.item()) == 0
    return ids.cpu().numpy(), lp.double().cpu().numpy()


class Row:
    """A row's order and exact running masses, in units of the largest's."""

    def __init__(self, x, t, k):
        x = np.asarray(x, np.float64)
        self.order = np.argsort(-x, kind="stable")
        self.order = self.order[np.isfinite(x[self.order])]
        if k > 0:
            self.order = self.order[:k]
        self.place = np.full(x.size, -1, np.int64)
        self.place[self.order] = np.arange(self.order.size)
        self.w = np.exp((x[self.order] - x[self.order[0]]).astype(np.longdouble) / np.longdouble(np.float32(t)))
        self.run = np.cumsum(self.w)

    def check(self, i, lp, u, p):
        n, at = self.order.size, int(self.place[i])
        assert at >= 0
        u, p = np.longdouble(np.float32(u)), np.longdouble(np.float32(p))
        off = 2.0 ** -29 + n * 2.0 ** -44 / self.run[-1]  # of the mass that top_p takes its share of
        lo = hi = n - 1
        if p < 1:
            cut = lambda share: min(n - 1, int(np.searchsorted(self.run, share * self.run[-1])))
            lo, hi = cut(max(p - off, 0)), cut(p + off)
        least, most = self.run[lo], self.run[hi]
        assert at <= hi
        off = 2.0 ** -29 + n * 2.0 ** -44 / least
        before, after = self.run[at] - self.w[at], self.run[at]
        assert before <= (u + off) * most and after >= (u - off) * least, (i, at, float(before), float(after), u)
        want = np.log(self.w[at] / least)
        room = 2.0 ** -24 * abs(want) + 2.0 ** -27 + n * 2.0 ** -44 / least + (most - least) / least
        # (a weight's own unit does not show: logprob is formed from the logit)
        assert abs(lp - want) <= room, (lp, float(want))


def flat_tail(v, depth, dt, at):
    """One token at 0, all others `depth` octaves of w lower at T = 1."""
    x = torch.full((v,), -depth * float(np.log(2.0)), device="cuda").to(DT[dt])
    x[at] = 0
    return x


def near_border(x, t, k):
    """Values of u next to the share of the largest token, and others."""
    row = Row(x.double().cpu().numpy(), t, k)
    f = np.float32(min(float(row.w[0] / row.run[-1]), 1 - 2.0 ** -24))
    us = [np.float32(0), np.float32(0.3), np.float32(1 - 2.0 ** -24)]
    lo = hi = f
    for _ in range(4):
        us += [lo, hi]
        lo, hi = np.nextafter(lo, np.float32(0)), min(np.nextafter(hi, np.float32(2)), np.float32(1 - 2.0 ** -24))
    return row, np.array(us, np.float32)


@pytest.mark.parametrize("v,dt", [(510001, "fp32"), (248320, "fp32"), (248320, "bf16"), (131072, "fp16"),
                                  (9001, "fp32")])
@pytest.mark.parametrize("depth", [12.3, 16.7, 20.9, 24.5, 28.1, 32.6, 36.2, 39.9954, 40.1, 43.3, 44.2, 47.0])
def test_flat_far_tail(gpu, v, dt, depth):
    x = flat_tail(v, depth, dt, v // 3)
    for t, k, p in ((1.0, 0, 1.0), (0.9, 0, 1.0), (1.0, v // 2, 1.0), (1.0, 0, 0.9999995), (1.0, v - 5, 0.99)):
        row, us = near_border(x, t, k)
        ids, lp = draw(x.expand(us.size, v).contiguous(), torch.as_tensor(us, device="cuda"), t, k, p)
        for i, l, u in zip(ids, lp, us):
            row.check(i, l, u, p)


def test_tail_at_a_sixteenth_of_a_unit_more_than_sixteen(gpu):
    """510,000 tokens of 16.05 units each, which count as 17."""
    x = torch.full((510001,), -27.722767, device="cuda")
    x[0] = 0
    row = Row(x.double().cpu().numpy(), 1.0, 0)
    us = (1 - np.arange(1, 16) * 2.0 ** -24).astype(np.float32)
    ids, lp = draw(x.expand(us.size, x.numel()).contiguous(), torch.as_tensor(us, device="cuda"), 1.0, 0, 1.0)
    for i, l, u in zip(ids, lp, us):
        row.check(i, l, u, 1.0)


@pytest.mark.parametrize("v,n", [(248320, 6), (16000, 400)])
def test_sloping_far_tails(gpu, v, n):
    """Tails that fall evenly from 14 to 60 octaves, one of them in narrow CTAs."""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = -0.6931 * (14 + 46 * torch.rand((n, v), generator=g, device="cuda"))
    x[:, 11] = 0
    x[:, 4000] = -9.0
    u = torch.linspace(0.9, 1 - 2.0 ** -24, n, device="cuda")
    for t, k, p in ((1.0, 0, 1.0), (1.0, v // 4, 0.99999), (1.1, 0, 0.9999)):
        ids, lp = draw(x, u, t, k, p)
        for r in range(0, n, max(1, n // 6)):
            Row(x[r].double().cpu().numpy(), t, k).check(ids[r], lp[r], float(u[r]), p)
