"""stv_rope against its definition in 64 bits (opkit.rope).

Tolerance per element, before the first run: half a step of the output type,
plus the fp32 arithmetic.  The phase's rounding to fp32 is at most 2^-25 of
half a turn (9.4e-8 rad), sine and cosine at most 2 units of 2^-24 (1.2e-7
each), two products and one sum 3 * 2^-24 (1.8e-7): together below 6e-7 times
(|a| + |b|) of the pair.  fp16 results below its normal range are off by up to
2^-25."""
import numpy as np
import pytest
import torch

import opkit
import speculative_tree_verify_bit_gb300 as stv

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def check(got, x, pos, rd, sections, theta, interleaved=False, inverse=False):
    want = opkit.rope(x.double().cpu().numpy(), pos.cpu().numpy().astype(np.int64), rd, sections, theta, interleaved,
                      inverse)
    g = got.double().cpu().numpy()
    assert np.array_equal(g[..., rd:], want[..., rd:])
    ax = np.abs(x.double().cpu().numpy()[..., :rd])
    h = rd // 2
    pair = np.tile(ax[..., :h] + ax[..., h:], 2)
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(want[..., :rd]) + 6e-7 * pair + (2.0 ** -25 if got.dtype ==
                                                                                  torch.float16 else 0)
    err = np.abs(g[..., :rd] - want[..., :rd])
    assert (err <= tol).all(), (err / tol).max()


def inputs(rows, hq, hkv, hd, dt, seed=1, axes=3, far=262144):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((rows, hq, hd), generator=g, device="cuda").to(DT[dt])
    k = torch.randn((rows, hkv, hd), generator=g, device="cuda").to(DT[dt])
    pos = torch.randint(0, far, (axes, rows), generator=g, device="cuda", dtype=torch.int32)
    return q, k, pos


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,hq,hkv,hd,rd,sections,inter", [
    (1, 24, 4, 256, 64, (12, 10, 10), False),
    (16, 24, 4, 256, 64, (12, 10, 10), True),
    (257, 24, 4, 256, 256, (48, 40, 40), False),
    (33, 3, 1, 128, 96, (16, 16, 16), True),
    (50, 5, 5, 64, 32, (16,), False),
    (7, 1, 1, 66, 30, (8, 7), False),     # no wide loads
    (5, 2, 1, 2, 2, (1,), False),
    (9, 7, 2, 512, 512, (64, 64, 64, 64), True),
    (40, 9, 3, 80, 48, (10, 8, 6), False),
])
def test_rope(gpu, dt, rows, hq, hkv, hd, rd, sections, inter):
    q, k, pos = inputs(rows, hq, hkv, hd, dt, axes=len(sections))
    spec = stv.make_rope(rd, sections, theta=1e6, interleaved=inter)
    for inverse in (False, True):
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        stv.stv_rope(spec, pos, q, qo, k, ko, inverse=inverse)
        check(qo, q, pos, rd, sections, 1e6, inter, inverse)
        check(ko, k, pos, rd, sections, 1e6, inter, inverse)


@pytest.mark.parametrize("dt", ["fp16", "fp32"])
def test_rope_strided_views_and_neighbours(gpu, dt):
    """q | k | v rows: the views are turned in place, v and the padding keep
    their bytes; and out of place into other columns of the same rows."""
    n, hq, hkv, hd, rd, sec = 45, 6, 2, 64, 32, (6, 5, 5)
    g = torch.Generator(device="cuda").manual_seed(2)
    row = torch.randn((n, (2 * hq + 3 * hkv) * hd + 8), generator=g, device="cuda").to(DT[dt])
    before = row.clone()
    pos = torch.randint(0, 9000, (3, n), generator=g, device="cuda", dtype=torch.int32)
    cut = lambda a, h: row[:, a * hd:(a + h) * hd].unflatten(1, (h, hd))
    q, k, qo, ko = cut(0, hq), cut(hq, hkv), cut(hq + 2 * hkv, hq), cut(2 * hq + 2 * hkv, hkv)
    spec = stv.make_rope(rd, sec)
    q0, k0 = q.clone(), k.clone()
    stv.stv_rope(spec, pos, q, qo, k, ko)
    check(qo, q0, pos, rd, sec, 1e4)
    check(ko, k0, pos, rd, sec, 1e4)
    assert torch.equal(row[:, :(hq + 2 * hkv) * hd], before[:, :(hq + 2 * hkv) * hd])
    stv.stv_rope(spec, pos, q, q, k, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    a = (hq + hkv) * hd
    assert torch.equal(row[:, a:a + hkv * hd], before[:, a:a + hkv * hd])
    assert torch.equal(row[:, -8:], before[:, -8:])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("n,heads,pad", [(1, 5, 0), (45, 6, 0), (45, 6, 24), (300, 1, 0)])
def test_rope_heads_side_by_side(gpu, dt, n, heads, pad):
    """q | k | v in each head: q and k turned in place; then q into v's place."""
    hd, rd, sec = 64, 48, (8, 8, 8)
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn((n, heads * 3 * hd + pad), generator=g, device="cuda").to(DT[dt])
    pos = torch.randint(0, 9000, (3, n), generator=g, device="cuda", dtype=torch.int32)
    x = row[:, :heads * 3 * hd].unflatten(1, (heads, 3, hd))
    q, k, v = x[:, :, 0], x[:, :, 1], x[:, :, 2]
    q0, k0, v0, rest = q.clone(), k.clone(), v.clone(), row[:, heads * 3 * hd:].clone()
    spec = stv.make_rope(rd, sec)
    stv.stv_rope(spec, pos, q, q, k, k)
    check(q, q0, pos, rd, sec, 1e4)
    check(k, k0, pos, rd, sec, 1e4)
    assert torch.equal(v, v0) and torch.equal(row[:, heads * 3 * hd:], rest)
    q1, k1 = q.clone(), k.clone()
    stv.stv_rope(spec, pos, q, v)
    check(v, q1, pos, rd, sec, 1e4)
    assert torch.equal(q, q1) and torch.equal(k, k1)


def test_rope_odd_strides_take_the_narrow_path(gpu):
    n, h, hd = 12, 3, 64
    buf = torch.randn((n, h, hd + 1), device="cuda", dtype=torch.float16)
    q = buf[..., :hd]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    spec = stv.make_rope(64, (32,))
    out = torch.empty((n, h, hd), device="cuda", dtype=torch.float16)
    stv.stv_rope(spec, pos, q, out)
    check(out, q, pos, 64, (32,), 1e4)
    wide = torch.empty_like(out)
    stv.stv_rope(spec, pos, q.contiguous(), wide)
    assert torch.equal(out, wide)


def test_rope_far_and_negative_positions(gpu):
    """Every int32 position keeps its phase (2^31 - 1 turns by a frequency of
    one radian), and -p undoes p."""
    pos = torch.tensor([[0, 1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, -7, 262143]], dtype=torch.int32, device="cuda")
    x = torch.randn((7, 2, 32), device="cuda")
    spec = stv.make_rope(32, (16,), theta=1.0)  # every pair turns by one radian a position
    y = torch.empty_like(x)
    stv.stv_rope(spec, pos, x, y)
    check(y, x, pos, 32, (16,), 1.0)


def test_rope_gradient(gpu):
    """The inverse call is the gradient: <g, R x> = <R^-1 g, x>, and against
    differences of the forward call in 32 bits."""
    q, _, pos = inputs(19, 4, 1, 64, "fp32", seed=5)
    g = torch.randn_like(q)
    spec = stv.make_rope(48, (8, 8, 8), interleaved=True)
    y, gx = torch.empty_like(q), torch.empty_like(q)
    stv.stv_rope(spec, pos, q, y)
    stv.stv_rope(spec, pos, g, gx, inverse=True)
    a, b = (g.double() * y.double()).sum().item(), (gx.double() * q.double()).sum().item()
    # each side is off by 6e-7 (|a| + |b|) an element, and partner terms: below 2e-6 |g| |x| in all
    assert abs(a - b) <= 2e-6 * g.double().norm().item() * q.double().norm().item()
    for e in (0, 1000, 4000):  # the map is linear: a difference at any step is exact up to rounding
        z = q.clone()
        z.view(-1)[e] += 0.5
        y2 = torch.empty_like(z)
        stv.stv_rope(spec, pos, z, y2)
        step = (z.view(-1)[e] - q.view(-1)[e]).item()
        num = (g.double() * (y2.double() - y.double())).sum().item() / step
        # the two outputs that change are each off by 6e-7 (|a| + |b|) <= 6e-6, both calls, over a step of 0.5
        assert abs(num - gx.view(-1)[e].item()) <= 1.2e-4


def test_rope_sixteen_bit_positions_past_32_bit_offsets(gpu):
    """Rows whose offsets pass 2^31 elements."""
    n, stride = 5, 1 << 29
    buf = torch.empty(n * stride + 64, device="cuda", dtype=torch.float16)
    x = buf.as_strided((n, 1, 64), (stride, 64, 1))
    src = torch.randn((n, 1, 64), device="cuda", dtype=torch.float16)
    x.copy_(src)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None] + 100
    stv.stv_rope(stv.make_rope(64, (32,)), pos, x, x)
    check(x, src, pos, 64, (32,), 1e4)


def test_rope_graph_and_stream(gpu):
    q, k, pos = inputs(16, 24, 4, 256, "bf16", seed=8)
    spec = stv.make_rope(64, (12, 10, 10))
    want = torch.empty_like(q)
    stv.stv_rope(spec, pos, q, want)
    qo = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stv.stv_rope(spec, pos, q, qo)
    side.synchronize()
    assert torch.equal(qo, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stv.stv_rope(spec, pos, q, qo)
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want * 2)  # doubling is exact


def test_rope_no_rows_and_one_view(gpu):
    spec = stv.make_rope(64, (12, 10, 10))
    e = torch.empty((0, 4, 64), device="cuda")
    stv.stv_rope(spec, torch.empty((3, 0), dtype=torch.int32, device="cuda"), e, e)
    q, k, pos = inputs(9, 4, 2, 64, "bf16", seed=11)
    both, alone = torch.empty_like(k), torch.empty_like(k)
    stv.stv_rope(spec, pos, q, torch.empty_like(q), k, both)
    stv.stv_rope(spec, pos, None, None, k, alone)
    assert torch.equal(both, alone)


def test_rope_python_refusals(gpu, monkeypatch):
    q, k, pos = inputs(4, 2, 1, 64, "fp16")
    spec = stv.make_rope(64, (12, 10, 10))
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        stv.stv_rope(spec, pos, q, None)
    with pytest.raises(ValueError):
        stv.stv_rope(spec, pos[:2].contiguous(), q, out)
    with pytest.raises(TypeError):
        stv.stv_rope(spec, pos, q, out.float())
    with pytest.raises(ValueError):
        stv.stv_rope(spec, pos, q, out[:3])
    with pytest.raises(TypeError):
        stv.stv_rope(spec, pos.long(), q, out)
    with pytest.raises(stv.StvError) as e:
        stv.stv_rope(spec, pos, q[:, :1], q[:, :1].as_strided((4, 1, 64), (128, 64, 1), 32))
    assert e.value.status == stv.STV_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        stv.stv_rope(spec, pos, q.cpu(), out)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)  # tensors on another device than the current one
    with pytest.raises(ValueError):
        stv.stv_rope(spec, pos, q, out)


@pytest.mark.parametrize("theta,rd", [(1.0, 64), (1e4, 64), (1e4, 256), (5e5, 128), (1e7, 96), (1e7, 256), (1e300, 8),
                                      (1e4, 2)])
def test_rope_phase_of_far_positions(gpu, theta, rd):
    """The phase at positions up to +-2^31, against frequencies formed to 70
    digits.  Rows of (1, 0) pairs come back as (cos, sin).  The phase is off by
    2^-26 of a turn when it is made an fp32 fraction of half a turn, 2^-32 when
    it is cut to 32 bits and 2^-34 from the frequency (2^-65 a position): below
    9.6e-8 rad; sine and cosine by at most 2 units of 2^-24 (1.2e-7); the
    products by 1 and 0 are exact."""
    from decimal import Decimal, localcontext

    pos = np.concatenate([2 ** 31 - 1 - np.arange(0, 4000, 97), -2 ** 31 + np.arange(0, 4000, 89),
                          2 ** 30 + np.arange(5), [0, 1, -1, 262143, 2 ** 24 + 1]])
    h, n = rd // 2, pos.size
    turns = np.empty((n, h))
    with localcontext() as c:
        c.prec = 70
        two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899863")
        for i in range(h):
            f = Decimal(theta) ** (Decimal(-2 * i) / Decimal(rd)) / two_pi
            turns[:, i] = [float((f * int(p)) % 1) for p in pos]
    x = torch.zeros((n, 1, rd), device="cuda")
    x[..., :h] = 1
    y = torch.empty_like(x)
    spec = stv.make_rope(rd, (h,), theta=theta)
    stv.stv_rope(spec, torch.as_tensor(pos.astype(np.int32), device="cuda")[None], x, y)
    got = y[:, 0].double().cpu().numpy()
    want = np.concatenate([np.cos(2 * np.pi * turns), np.sin(2 * np.pi * turns)], 1)
    assert np.abs(got - want).max() <= 9.6e-8 + 1.2e-7, np.abs(got - want).max()
