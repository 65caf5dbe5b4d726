"""stv_page_extend where positions come near the end of 32 bits."""
import numpy as np
import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from drafterkit import PAGE, dev

pytestmark = pytest.mark.gpu

MOST = 2**31 - 1


@pytest.mark.parametrize("rows", [8, 5000])
@pytest.mark.parametrize("ctx,new,fits", [(MOST - 5, 5, True), (MOST - 4, 5, False), (MOST, 1, False),
                                          (MOST - 4096, 4000, True), (MOST, 0, True)])
def test_positions_stay_within_32_bits(gpu, ctx, new, fits, rows):
    """A sequence whose table (the pool's pages named again and again) is long enough for more
    tokens than 32 bits count."""
    stride = 2**23 + 64
    table = torch.arange(stride, dtype=torch.int32, device="cuda").remainder_(7)[None].contiguous()
    pool = stv.PagePool(torch.ones(7, dtype=torch.int32, device="cuda"), table.clone(), dev([stride]))
    start, status = dev([-9, -9]), dev([0])
    maps = torch.full((3, rows), -9, dtype=torch.int32, device="cuda")
    stv.stv_page_extend(pool, None, dev([new]), dev([ctx]), start, *maps, dev_status=status)
    want = np.full((3, rows), -1, np.int64)
    if fits and new <= rows:
        pos = ctx + np.arange(new, dtype=np.int64)
        want[:, :new] = np.zeros(new), pos, pos // PAGE % 7 * PAGE + pos % PAGE
        assert status.item() == 0 and start.tolist() == [0, new]
    else:
        assert status.item() == (stv.STV_DEV_BAD_ROW if fits else stv.STV_DEV_BAD_SEQ) and start.tolist() == [0, 0]
    assert np.array_equal(maps.cpu().numpy(), want)
    assert torch.equal(pool.tables, table) and pool.counts.item() == stride
