"""stv_paged_attn with o in the other half of q's heads."""
import pytest
import torch

from drafterkit import Drafter
from test_gpu_paged_attn import call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("hd,new,pad", [(128, 1, 0), (64, 40, 0), (256, 33, 8), (128, 90, 1)])
def test_o_between_the_heads_of_q(gpu, hd, new, pad, order):
    d = Drafter([500, 77 + new], 2, hd, torch.bfloat16, seed=hd)
    entries = [(0, 500 - new, 0, new), (1, 77, new, new)]
    both = torch.full((2 * new, 8, 2 * hd + pad), 3.0, dtype=torch.bfloat16, device="cuda")
    q, o = (both[:, :, i * hd:(i + 1) * hd] for i in (order, 1 - order))
    q.copy_(d.rows(2 * new, 8))
    kept = q.clone()
    check(d, kept, entries, call(d, q, entries, o=o))
    assert torch.equal(q, kept) and (both[:, :, 2 * hd:] == 3.0).all()
