"""stv_tree_accept_probs handing over to stv_kv_commit: what was accepted by
probabilities is what the target's cache keeps."""
import numpy as np
import pytest
import torch

import oracle
import speculative_tree_verify_bit_gb300 as stv
from drafterkit import accept, dev
from roundkit import Round

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("drafts", ["replaced", "distinct", "certain"])
@pytest.mark.parametrize("ctx,t", [([1024], 16), ([250, 13, 4000], 16), ([255, 511], 21)])
def test_accepted_rows_are_committed(gpu, ctx, t, drafts):
    rng = np.random.default_rng(t + len(ctx))
    n, vocab = len(ctx), 60
    rounds = [Round(ctx, t, seed=500 + l) for l in range(2)]
    base = rounds[0]
    for r in rounds[1:]:
        r.parent, r.tables = base.parent, base.tables
    layers, caches = [r.gpu_cache() for r in rounds], [r.oracle_cache() for r in rounds]
    P, Q = (np.float32(rng.dirichlet(np.full(vocab, 0.3), n * t)) for _ in range(2))
    ids = rng.integers(0, vocab, (n, t))
    for s in range(n):  # many likely children, so that paths are long
        for i in range(1, t):
            if rng.random() < 0.7:
                ids[s, i] = int(np.argmax(P[s * t + base.parent[s][i]]))
    u = np.float32(rng.random((n, t)) * 0.999)
    nc, path, out = dev([0] * n), dev(np.zeros((n, t))), dev(np.zeros((n, t)))
    ctx_dev, status = dev(ctx), dev([0])
    f32 = lambda x: torch.as_tensor(x, device="cuda")
    stv.stv_tree_accept_probs(dev(base.parent), dev(ids), f32(P), None if drafts == "certain" else f32(Q), f32(u), nc, path, out,
                              distinct=drafts == "distinct", dev_status=status)
    stv.stv_kv_commit(base.shape, layers, base.seqs, t, nc, path, ctx_dev=ctx_dev, dev_status=status)
    assert status.item() == 0
    want_n, want_path = np.zeros(n, np.int32), np.zeros((n, t), np.int32)
    for s in range(n):
        rs = slice(s * t, (s + 1) * t)
        way, _, gap = accept(base.parent[s], ids[s], P[rs].astype(np.float64),
                             None if drafts == "certain" else Q[rs].astype(np.float64), u[s].astype(np.float64),
                             drafts == "distinct")
        assert gap > 1e-11
        want_n[s], want_path[s, :len(way)] = len(way), way
    assert n == 1 or drafts == "certain" or want_n.max() > 2  # (the 64-bit form: some path is long)
    assert nc.cpu().numpy().tolist() == want_n.tolist()
    assert ctx_dev.cpu().numpy().tolist() == [c + int(m) for c, m in zip(ctx, want_n)]
    for layer, cache in zip(layers, caches):
        oracle.kv_commit(cache, base.tables, ctx, want_n, want_path, t)
        assert np.array_equal(layer.pool.cpu().numpy(), cache.pool)


def test_a_refused_sequence_commits_nothing(gpu):
    """A sequence whose probabilities are bad has n_commit 0, which commit refuses for it alone."""
    t = 8
    r = Round([300, 40], t, seed=9)
    layer = r.gpu_cache()
    before = layer.pool.clone()
    p = torch.full((2 * t, 12), 1 / 12, device="cuda")
    p[t:] = float("nan")
    parent = torch.as_tensor(np.stack(r.parent), dtype=torch.int32, device="cuda")
    nc, path, out = dev([9, 9]), dev(np.zeros((2, t))), dev(np.zeros((2, t)))
    ctx, status = dev([300, 40]), dev([0])
    stv.stv_tree_accept_probs(parent, dev(np.zeros((2, t))), p, None, torch.full((2, t), 0.9, device="cuda"), nc, path, out,
                              dev_status=status)
    assert status.item() == stv.STV_DEV_BAD_SAMPLE and nc.tolist() == [1, 0]
    stv.stv_kv_commit(r.shape, [layer], r.seqs, t, nc, path, ctx_dev=ctx, dev_status=status)
    assert status.item() == stv.STV_DEV_BAD_SAMPLE | stv.STV_DEV_BAD_COMMIT
    assert ctx.tolist() == [301, 40] and torch.equal(layer.pool, before)
