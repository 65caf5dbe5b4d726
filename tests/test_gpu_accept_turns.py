"""stv_tree_accept_probs where many rejections follow one another: every turn
hands numbers from one thread to a cluster and back."""
import numpy as np
import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from drafterkit import accept, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("distinct", [False, True])
@pytest.mark.parametrize("n", [9, 19, 38, 76, 152])
def test_a_node_whose_children_are_all_rejected(gpu, n, distinct):
    """31 rejections at one node of equal sequences, in clusters of 16 down to 1 CTA: every
    sequence has the 64-bit form's answer, in every one of 20 calls."""
    rng = np.random.default_rng(31)
    t, vocab = 32, 65536 + 77
    x = np.exp(2 * rng.normal(size=(2, vocab)))
    kids = rng.choice(vocab, t - 1, replace=False)
    x[0, kids] = 0  # none of them is the target's
    x[0, 11] = x[0].sum() * 0.5
    x /= x.sum(1, keepdims=True)
    p, q = (torch.as_tensor(r, dtype=torch.float32, device="cuda") for r in x)
    parent = np.array([-1] + [0] * (t - 1))
    ids = np.concatenate([[0], kids])
    u = np.float32(0.3 + 0.69 * rng.random(t))
    rows = [r.repeat(n * t, 1) for r in (p, q)]
    P, Q = (np.tile(r.double().cpu().numpy(), (t, 1)) for r in (p, q))
    path, out, gap = accept(parent, ids, P, Q, u.astype(np.float64), distinct)
    assert path == [0] and gap > 1e-11
    a = [dev(np.tile(parent, (n, 1))), dev(np.tile(ids, (n, 1))), *rows, dev(np.tile(u, (n, 1)), torch.float32)]
    for _ in range(20):
        nc, pa, got = (torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((n,), (n, t), (n, t)))
        stv.stv_tree_accept_probs(*a, nc, pa, got, distinct=distinct)
        assert (nc == 1).all() and (pa[:, 0] == 0).all() and (pa[:, 1:] == -1).all()
        assert (got[:, 0] == out[0]).all() and (got[:, 1:] == -1).all()
