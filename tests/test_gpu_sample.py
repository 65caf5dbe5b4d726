"""stv_sample against its definition in 64 bits (opkit.sample).

Ids must be equal, except where u falls within 2^-28 of the kept mass of a
border between two tokens: weights carry a relative error below 2^-28, so a
share f of the mass is off by at most f (1 - f) 2^-27 <= 2^-29, at the cut of
top_p and at the draw.  logprob is off by the fp32 rounding, 2^-24 of its
value, and the errors of the masses and their logarithms, 2^-27."""
import numpy as np
import pytest
import torch

import opkit
import speculative_tree_verify_bit_gb300 as stv

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def draw(logits, u, t=None, k=None, p=None, m=None, rpp=1, status=None):
    n = logits.shape[0]
    ids = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((n,), 7.0, device="cuda")
    f = lambda v, dt: None if v is None else torch.as_tensor(np.asarray(v, dt), device="cuda")
    stv.stv_sample(logits, u, ids, lp, f(t, np.float32), f(k, np.int32), f(p, np.float32), f(m, np.float32), rpp,
                   dev_status=status)
    return ids.cpu().numpy(), lp.cpu().numpy()


def check(logits, u, t=None, k=None, p=None, m=None, rpp=1):
    ids, lp = draw(logits, u, t, k, p, m, rpp)
    lp = lp.astype(np.float64)  # the differences below in 64 bits
    x, us = logits.double().cpu().numpy(), u.cpu().numpy()
    at = lambda v, r, d: d if v is None else v[r // rpp]
    for r in range(len(us)):
        i, l, gap = opkit.sample(x[r], us[r], at(t, r, 1.0), int(at(k, r, 0)), at(p, r, 1.0), at(m, r, 0.0))
        if gap > 2.0 ** -28:
            assert ids[r] == i, (r, ids[r], i, gap)
            assert lp[r] == l or abs(lp[r] - l) <= 2.0 ** -24 * abs(l) + 2.0 ** -27, (r, lp[r], l)


def rows(n, v, dt, seed=0, sigma=2.5, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = (sigma * torch.randn((n, v + pad), generator=g, device="cuda")).to(DT[dt])
    return buf[:, :v], torch.rand(n, generator=g, device="cuda")


SETS = [
    dict(),
    dict(t=[0.7]),
    dict(t=[0.0]),
    dict(k=[1]),
    dict(k=[50], t=[0.8]),
    dict(p=[0.9]),
    dict(p=[0.0]),
    dict(m=[0.05]),
    dict(m=[1.0]),
    dict(t=[1.3], k=[1000], p=[0.95], m=[0.02]),
    dict(t=[5.0], p=[0.999]),
    dict(t=[1e-3]),
    dict(t=[1e-30]),
    dict(t=[1e6], p=[0.5]),
    dict(k=[100000000], p=[1.5]),
    dict(k=[-3]),
    dict(p=[1e-40]),
    dict(p=[0.99999994]),
    dict(m=[1e-40]),
    dict(t=[0.3], m=[1e-6]),
    dict(k=[2], p=[0.6], m=[0.9]),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("n,v,pad", [(1, 1, 0), (3, 2, 1), (5, 31, 0), (4, 1000, 3), (7, 32003, 5), (2, 248320, 0)])
def test_sample(gpu, dt, n, v, pad):
    logits, u = rows(n, v, dt, seed=v + n, pad=pad)
    for a in SETS:
        check(logits, u, rpp=n, **a)


@pytest.mark.parametrize("v", [40, 5000, 70001, 262144, 524288])
def test_sample_flat_rows(gpu, v):
    """Equal logits, two values, and a slope smaller than a bin: too many
    tokens around every cut to gather at once, and ties told apart by index."""
    x = torch.zeros((3, v), device="cuda")
    x[1, ::3] = 0.25
    x[2] = torch.linspace(-1e-3, 1e-3, v, device="cuda")
    u = torch.tensor([0.4, 0.77, 0.123], device="cuda")
    for a in (dict(), dict(k=[v // 2 + 1]), dict(p=[0.6]), dict(m=[0.999]), dict(k=[v // 2], p=[0.5], m=[0.5], t=[2.0]),
              dict(t=[100.0], p=[0.3])):
        check(x, u, rpp=3, **a)
    check(x.half(), u, rpp=3, p=[0.9], k=[v - 1])


def test_sample_extreme_values(gpu):
    big = torch.full((4, 3000), -3e38, device="cuda")
    big[0, 17] = 3e38
    big[1, 5] = 0.0
    big[2] = torch.linspace(-60000, 60000, 3000, device="cuda")
    big[3, 100:200] = 1e-40
    u = torch.tensor([0.0, 0.5, 0.99999994, 0.5], device="cuda")
    for a in (dict(), dict(t=[1e4]), dict(p=[0.5], k=[7]), dict(t=[2.0 ** 60]), dict(t=[2.0 ** -100])):
        check(big, u, rpp=4, **a)
    # max - x over T = 3e38 has no fp32 form: such a temperature is refused
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in (3e38, 2.0 ** 61, 2.0 ** -101, 1e-45):
        status.zero_()
        assert (draw(big, u, t=[t], rpp=4, status=status)[0] == -1).all()
        assert int(status.item()) == stv.STV_DEV_BAD_SAMPLE
    zeros = torch.zeros((1, 64), device="cuda")
    zeros[0, ::2] = -0.0  # one value
    check(zeros, torch.tensor([0.51], device="cuda"), k=[33])


def test_sample_masks(gpu):
    """-inf takes no part: most of a row, all but one token, the first and last."""
    logits, u = rows(6, 5003, "fp16", seed=3)
    logits[0, torch.rand(5003, device="cuda") < 0.95] = -float("inf")
    logits[0, 40] = 1
    logits[1] = -float("inf")
    logits[1, 5002] = -3.0
    logits[2] = -float("inf")
    logits[2, 0] = -65504.0
    logits[3, 1:] = -65504.0  # the type's lowest value is not a mask
    logits[4, :2500] = -float("inf")
    for a in SETS:
        check(logits, u, rpp=6, **a)
    ids, lp = draw(logits, u, k=[100000], rpp=6)
    assert ids[1] == 5002 and lp[1] == 0 and ids[2] == 0


def test_sample_bad_rows_are_reported_and_alone(gpu):
    logits, u = rows(8, 700, "fp32", seed=4)
    want, _ = draw(logits, u)
    logits[1] = -float("inf")
    logits[2, 650] = float("nan")
    logits[3, 2] = float("inf")
    u[4] = 1.0
    u[5] = float("nan")
    u[6] = -0.25
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, lp = draw(logits, u, status=status)
    assert int(status.item()) == stv.STV_DEV_BAD_SAMPLE
    assert ids.tolist() == [want[0], -1, -1, -1, -1, -1, -1, want[7]]
    assert np.isneginf(lp[1:7]).all() and np.isfinite(lp[[0, 7]]).all()
    for a in (dict(t=[-1.0]), dict(t=[float("nan")]), dict(t=[float("inf")]), dict(p=[-0.1]), dict(p=[float("nan")]),
              dict(m=[-0.1]), dict(m=[1.5]), dict(m=[float("nan")])):
        status.zero_()
        ids, _ = draw(logits[:1], u[:1], status=status, **a)
        assert ids[0] == -1 and int(status.item()) == stv.STV_DEV_BAD_SAMPLE, a
    draw(logits[:1], u[:1], t=[-1.0])  # no status word: nothing to report to


def test_sample_parameters_per_request(gpu):
    """rows_per_param rows share their entry; the last group may be short."""
    logits, u = rows(11, 9001, "bf16", seed=6)
    check(logits, u, t=[0.0, 0.6, 1.1], k=[0, 5, 40], p=[0.5, 1.0, 0.8], m=[0.0, 0.0, 0.1], rpp=4)


@pytest.mark.parametrize("n", [1, 8, 30, 75, 200, 520])
def test_sample_row_counts(gpu, n):
    logits, u = rows(n, 20011, "fp16", seed=n)
    check(logits, u, t=[0.9], p=[0.9], rpp=n)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("v", [1, 130, 2000, 16384])
def test_sample_many_short_rows(gpu, dt, v):
    """More short rows than SMs hold wide CTAs for: one narrow CTA per row.
    Against the definition, and the same as the rows get a few at a time."""
    n = 420
    logits, u = rows(n, v, dt, seed=v, pad=3)
    logits[5:9] = 0.5                      # flat
    logits[9, : v // 2] = -float("inf")
    logits[10] *= 0.01
    kw = [dict(), dict(t=[0.7], p=[0.9]), dict(k=[40], p=[0.95], m=[0.01]), dict(k=[700], t=[2.0]), dict(t=[3.0], p=[0.99]),
          dict(m=[0.3]), dict(t=[0.0])]
    for a in kw:
        ids, lp = draw(logits, u, rpp=n, **a)
        few, lp2 = draw(logits[:40], u[:40], rpp=40, **a)
        assert np.array_equal(ids[:40], few) and np.array_equal(lp[:40], lp2)
    check(logits[:n], u, rpp=n, **kw[v % len(kw)])
    check(logits[:n], u, rpp=n, t=[1.5], p=[0.97])


def test_sample_does_not_depend_on_the_batch(gpu):
    """A row's token and logprob are the same alone, in a batch, twice, and
    wherever the row starts."""
    logits, u = rows(160, 30000, "fp32", seed=9)
    kw = dict(t=[0.9], k=[0], p=[0.92], m=[0.001])
    ids, lp = draw(logits, u, rpp=160, **kw)
    again, lp2 = draw(logits, u, rpp=160, **kw)
    assert np.array_equal(ids, again) and np.array_equal(lp, lp2)
    for r in (0, 77, 159):
        one, l = draw(logits[r:r + 1].contiguous(), u[r:r + 1], **kw)
        assert one[0] == ids[r] and l[0] == lp[r]
    off = torch.empty((160, 30003), device="cuda")
    off[:, 3:] = logits
    moved, lp3 = draw(off[:, 3:], u, rpp=160, **kw)
    assert np.array_equal(ids, moved) and np.array_equal(lp, lp3)


def test_sample_shares(gpu):
    """Evenly spaced u draw every token for its share of the kept mass."""
    n = 4096
    x = torch.tensor([0.0, 1.5, -float("inf"), 1.5, 3.0, -2.0, 0.5], device="cuda").expand(n, 7).contiguous()
    u = (torch.arange(n, device="cuda") + 0.5) / n
    ids, lp = draw(x, u, t=[1.2], rpp=n)
    w = np.exp(x[0].double().cpu().numpy() / np.float64(np.float32(1.2)))
    assert np.abs(np.bincount(ids, minlength=7) / n - w / w.sum()).max() <= 1.0 / n
    assert np.abs(np.exp(lp.astype(np.float64)) - (w / w.sum())[ids]).max() <= 1e-6


def test_sample_graph_stream_and_large_offsets(gpu):
    logits, u = rows(16, 248320, "bf16", seed=12)
    ids = torch.zeros(16, dtype=torch.int32, device="cuda")
    t = torch.full((1,), 0.8, device="cuda")
    want, _ = draw(logits, u, t=[0.8], rpp=16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stv.stv_sample(logits, u, ids, temperature=t, rows_per_param=16)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), want)
    u.copy_(torch.rand(16, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids2 = torch.zeros_like(ids)
    stv.stv_sample(logits, u, ids2, temperature=t, rows_per_param=16, stream=side)
    side.synchronize()
    assert torch.equal(ids, ids2)
    stride = (1 << 31) + 8  # the second row's offset passes 32 bits
    far = torch.empty(stride + 5000, device="cuda", dtype=torch.float16).as_strided((2, 5000), (stride, 1))
    near, u2 = rows(2, 5000, "fp16", seed=13)
    far.copy_(near)
    a, b = draw(far, u2), draw(near, u2)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_sample_no_rows(gpu):
    e = torch.empty(0, device="cuda")
    stv.stv_sample(torch.empty((0, 100), device="cuda"), e, torch.empty(0, dtype=torch.int32, device="cuda"), e)


def test_sample_smallest_u_and_largest(gpu):
    """u of 0, the least subnormal and the largest below 1, over a row whose
    last token in the order has next to no mass."""
    x = torch.tensor([[0.0, 20.0, -20.0, 5.0]], device="cuda").expand(4, 4).contiguous()
    u = torch.tensor([0.0, 1e-45, 1.1754944e-38, 0.99999994], device="cuda")
    check(x, u, rpp=4)
    check(x, u, rpp=4, t=[30.0])


@pytest.mark.parametrize("v", [7, 1901, 70001])
def test_sample_negative_zeros(gpu, v):
    """u, top_p, min_p and T of -0 are zeros."""
    logits, _ = rows(3, v, "fp32", seed=21)
    u0, u1 = torch.zeros(3, device="cuda"), torch.full((3,), -0.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for a in (dict(), dict(k=[5]), dict(p=[0.0]), dict(t=[0.7], p=[0.9], m=[0.0]), dict(t=[0.0])):
        neg = {key: [-x if x == 0 else x for x in val] if key != "k" else val for key, val in a.items()}
        want, got = draw(logits, u0, rpp=3, **a), draw(logits, u1, rpp=3, status=status, **neg)
        assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])
        check(logits, u1, rpp=3, **neg)
    check(logits, torch.tensor([0.2, 0.6, 0.97], device="cuda"), rpp=3, p=[-0.0])
    assert int(status.item()) == 0


@pytest.mark.parametrize("v", [60000, 248320])
def test_sample_long_tails(gpu, v):
    """A few heavy tokens over a wide tail: the cuts lie far down the order."""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn((12, v), generator=g, device="cuda")
    x[:, 7::9001] += 9.0
    x[6:] *= 0.2
    u = torch.linspace(0.02, 0.9999, 12, device="cuda")
    for a in (dict(), dict(p=[0.97]), dict(k=[v // 3], p=[0.8]), dict(k=[5000]), dict(m=[0.003]), dict(k=[1900]),
              dict(t=[0.4], p=[0.9999]), dict(k=[v - 2], m=[1e-4])):
        check(x, u, rpp=12, **a)
    check(x.bfloat16(), u, rpp=12, p=[0.99])


def test_sample_python_refusals(gpu, monkeypatch):
    logits, u = rows(4, 100, "fp32")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        stv.stv_sample(logits.t(), u, ids)
    with pytest.raises(ValueError):
        stv.stv_sample(logits, u[:3], ids)
    with pytest.raises(ValueError):
        stv.stv_sample(logits, u, ids, temperature=torch.ones(2, device="cuda"))
    with pytest.raises(TypeError):
        stv.stv_sample(logits, u, ids.long())
    with pytest.raises(TypeError):
        stv.stv_sample(logits.double(), u, ids)
    with pytest.raises(ValueError):
        stv.stv_sample(logits, u, ids, rows_per_param=0)
    with pytest.raises((TypeError, ValueError)):
        stv.stv_sample(logits, u.cpu(), ids)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)  # tensors on another device than the current one
    with pytest.raises(ValueError):
        stv.stv_sample(logits, u, ids)
