"""stv_paged_attn where many small weights count: fp16 P carries a factor of
2^7, so that what a key adds is kept down to 2^-32 of its row's largest."""
import numpy as np
import pytest
import torch

from drafterkit import PAGE, Drafter, attention
from test_gpu_paged_attn import BF16, FP16, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_a_long_flat_tail_counts(gpu, n, hd, dtype):
    """One key far ahead of 60,000 equal ones, each 2^-26 of it: together 9e-4."""
    length, hkv, g = 60000, 2, 3
    d = Drafter([length], hkv, hd, dtype, seed=22, fill=0.0)
    for e in range(-(-length // PAGE)):
        page = int(d.pool.tables[0, e])
        d.data[page, :, 0], d.data[page, :, 1] = 0, 1.0
    first = int(d.pool.tables[0, 0])
    d.data[first, :, 0, 7], d.data[first, :, 1, 7] = 1.0, 0.0
    q = torch.ones((n, hkv * g, hd), dtype=dtype, device="cuda")
    got = call(d, q, [(0, length - n, 0, n)], scale=26 * np.log(2.0) / hd).double()
    tail = (length - n + torch.arange(1, n + 1, device="cuda").double() - 1) * 2.0 ** -26
    want = (tail / (1 + tail))[:, None, None]
    # P (2^-26 and 1) is exact in both types, the result rounded; 26 ln 2 log2(e) / hd in fp32, and fp32
    # sums of up to 60,000 equal numbers
    tol = want * (torch.finfo(dtype).eps / 2 + 26 * 2.0 ** -22 + length * 2.0 ** -24)
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_long_contexts_within_what_is_kept(gpu, n, hd, dtype):
    """20,001 keys, most of them far below the row's largest, against the bound of what the kernels keep."""
    ctx, hkv, g = 20001 - n, 2, 4
    d = Drafter([ctx + n], hkv, hd, dtype, seed=23)
    q = 3 * d.rows(n, hkv * g)
    entries = [(0, ctx, 0, n)]
    want, tol = attention(d, q, entries)
    keys = ctx + n
    most = d.keys(0, keys)[:, :, 1].abs().amax((0, 2)).repeat_interleave(g)[None, :, None]
    if dtype == FP16:
        # `attention` allows 2^-25 of V's largest a key.  With P = 2^(s - m + 7), the largest at least 2^7, half
        # a step below the normal numbers is 2^-25: 2^-32 of the row's largest, whose share is 1 at most
        tol = tol + keys * (2.0 ** -32 - 2.0 ** -25) * most
        assert (tol > 0).all()
    got = call(d, q, entries).double()
    err = (got - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
