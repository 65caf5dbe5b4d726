"""Failure detection of stv_paged_attn without a GPU fault."""
import time

import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from drafterkit import Drafter, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("hd,new", [(128, 1), (64, 1), (128, 90), (64, 20), (256, 30)])
def test_waits_run_out_and_the_context_stays_usable(gpu, hd, new, wide):
    """The kernels with their copies of K and V withheld: every wait for one gives up, whatever was under way
    (Q by TMA, or by plain loads) is waited for, and the next call is right."""
    d = Drafter([3000, 200, 700], 2, hd, torch.bfloat16, seed=hd + new)
    lens = [3000, 200, 700]
    q = torch.zeros((3 * new, 8, hd + (0 if wide else 1)), dtype=torch.bfloat16, device="cuda")[:, :, :hd]
    q.copy_(d.rows(3 * new, 8))
    shape, spec = stv.make_row_shape(8, 2, hd, torch.bfloat16), stv.make_attn()
    ws = torch.zeros(stv.stv_paged_attn_workspace_bytes(shape, new), dtype=torch.uint8, device="cuda")
    o, status = torch.zeros((3 * new, 8, hd), dtype=torch.bfloat16, device="cuda"), dev([0])
    args = (shape, spec, d.layer, d.pool, None, dev([n - new for n in lens]), dev([0, new, 2 * new, 3 * new]), new, q)
    stv.stv_paged_attn(*args, o, ws, dev_status=status)
    want = o.clone()
    assert status.item() == 0
    t0 = time.monotonic()
    stv.stv_paged_attn_timeout_test(*args, o, ws, dev_status=status)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 30.0
    assert status.item() == stv.STV_DEV_TIMEOUT
    status.zero_()
    stv.stv_paged_attn(*args, o, ws, dev_status=status)
    assert status.item() == 0 and torch.equal(o, want)
