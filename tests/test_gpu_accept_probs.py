"""stv_tree_accept_probs against its 64-bit form, row by row, and against
what it is for: what is committed is distributed as the target."""
import numpy as np
import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from drafterkit import accept, dev

pytestmark = pytest.mark.gpu

KINDS = ["replaced", "distinct", "certain"]
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def tree(rng, t, kind):
    if kind == "chain":
        return np.arange(-1, t - 1)
    if kind == "star":
        return np.array([-1] + [0] * (t - 1))
    return np.array([-1] + [int(rng.integers(0, max(1, (i + 1) // 2))) for i in range(1, t)])


def rows(rng, n, vocab, dtype, stride, sharp, shift=0):
    """Probability rows of a softmax, some entries exactly 0, any distance apart."""
    x = rng.normal(size=(n, vocab)) * sharp
    x[rng.random((n, vocab)) < 0.2] = -np.inf
    x[:, 0] = 0
    x = np.exp(x - x.max(1, keepdims=True))
    x /= x.sum(1, keepdims=True)
    buf = torch.full((n * stride + shift,), 9.0, dtype=dtype, device="cuda")[shift:].view(n, stride)
    buf[:, :vocab] = torch.as_tensor(x, device="cuda").to(dtype)
    return buf[:, :vocab]


def call(parent, ids, p, q, u, distinct=False, status=None):
    n, t = parent.shape
    out = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((n,), (n, t), (n, t))]
    stv.stv_tree_accept_probs(dev(parent), dev(ids), p, q, dev(u, torch.float32), *out, distinct=distinct, dev_status=status)
    return [o.cpu().numpy() for o in out]


@pytest.mark.parametrize("drafts", KINDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("n,t,vocab,pad,shift,shape", [
    (3, 1, 1, 0, 0, "chain"), (5, 8, 17, 0, 0, "tree"), (4, 32, 1000, 3, 1, "star"), (6, 16, 4097, 0, 0, "tree"),
    (2, 32, 33000, 8, 0, "chain"), (1, 9, 131071, 1, 3, "tree"), (40, 12, 9001, 0, 0, "star"),
    (1, 7, 524288, 0, 0, "star")])
def test_rows_of_every_kind(gpu, n, t, vocab, pad, shift, shape, dtype, drafts):
    rng = np.random.default_rng(t + vocab)
    p = rows(rng, n * t, vocab, dtype, vocab + pad, 2.0, shift)
    q = None if drafts == "certain" else rows(rng, n * t, vocab, dtype, vocab + pad + (5 if n == 4 else 0), 1.5, shift)
    P = p.double().cpu().numpy()
    Q = None if q is None else q.double().cpu().numpy()
    parent = np.stack([tree(rng, t, shape) for _ in range(n)])
    ids = np.zeros((n, t), np.int64)
    for s in range(n):
        for i in range(1, t):  # likely tokens, any token, and now and then none
            row = (Q if Q is not None and rng.random() < 0.7 else P)[s * t + parent[s, i]]
            ids[s, i] = rng.choice(vocab, p=row / row.sum()) if rng.random() < 0.8 else rng.integers(-1, vocab + 1)
    u = np.float32(rng.random((n, t)) * 0.9999)
    u[rng.random((n, t)) < 0.05] = 0.0
    n_commit, path, out = call(parent, ids, p, q, u, drafts == "distinct")
    seen = 0
    for s in range(n):
        rs = slice(s * t, (s + 1) * t)
        want_path, want_out, gap = accept(parent[s], ids[s], P[rs], None if Q is None else Q[rs], u[s].astype(np.float64),
                                          drafts == "distinct")
        m = len(want_path)
        if gap < 1e-11:  # both forms round: 2^-60 a token here (F q: 2^-46 of it), 2^-53 an operation there
            continue
        seen += 1
        assert n_commit[s] == m and path[s, :m].tolist() == want_path and out[s, :m].tolist() == want_out
        assert (path[s, m:] == -1).all() and (out[s, m:] == -1).all()
    assert seen >= n - 1


@pytest.mark.parametrize("drafts", KINDS)
def test_equal_rows_accept_and_one_hot_rows(gpu, drafts):
    """p = q accepts its own drafts whatever u; a one-hot target commits its token and nothing else."""
    rng = np.random.default_rng(5)
    t, vocab = 6, 500
    p = rows(rng, t, vocab, torch.float32, vocab, 1.0)
    parent = tree(rng, t, "chain")[None]
    if drafts != "certain":
        ids = np.array([[0] + [int(rng.choice(np.nonzero(p[i].cpu().numpy())[0])) for i in range(t - 1)]])
        n_commit, path, out = call(parent, ids, p, p, np.full((1, t), 1 - 2.0 ** -24, np.float32), drafts == "distinct")
        assert n_commit[0] == t and out[0, :-1].tolist() == ids[0, 1:].tolist()
    hot = torch.zeros((t, vocab), device="cuda")
    tok = rng.integers(0, vocab, t)
    hot[torch.arange(t), torch.as_tensor(tok, device="cuda")] = 1.0
    ids = np.array([[0, tok[0], tok[1], (tok[2] + 1) % vocab, 3, 4]])
    q = None if drafts == "certain" else torch.full((t, vocab), 1.0 / vocab, device="cuda")
    n_commit, path, out = call(parent, ids, hot, q, np.float32(rng.random((1, t))), drafts == "distinct")
    assert n_commit[0] == 3 and out[0, :3].tolist() == tok[:3].tolist()


@pytest.mark.parametrize("drafts", KINDS)
def test_committed_tokens_are_distributed_as_the_target(gpu, drafts):
    """40,000 sequences of one node and three drafted children on 6 tokens: the
    first committed token's frequencies, each within 6 standard deviations."""
    rng = np.random.default_rng(6)
    n, t, vocab = 40000, 4, 6
    target, draft = np.array([0.05, 0.3, 0.0, 0.25, 0.3, 0.1]), np.array([0.4, 0.1, 0.2, 0.05, 0.15, 0.1])
    p = torch.tensor(np.tile(target, (n * t, 1)), dtype=torch.float32, device="cuda")
    q = torch.tensor(np.tile(draft, (n * t, 1)), dtype=torch.float32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    kids = torch.multinomial(q[:n], t - 1, replacement=drafts != "distinct", generator=g).cpu().numpy()
    if drafts == "certain":  # any fixed rule
        kids[:] = [0, 1, 4]
    ids = np.concatenate([np.zeros((n, 1), np.int64), kids], 1)
    parent = np.tile(tree(rng, t, "star"), (n, 1))
    u = torch.rand((n, t), generator=g, device="cuda").cpu().numpy()
    n_commit, path, out = call(parent, ids, p, None if drafts == "certain" else q, u, drafts == "distinct")
    freq = np.bincount(out[:, 0], minlength=vocab) / n
    assert (np.abs(freq - target) <= 6 * np.sqrt(target * (1 - target) / n)).all(), freq
    assert freq[2] == 0


@pytest.mark.parametrize("what,bit", [("nan", stv.STV_DEV_BAD_SAMPLE), ("negative", stv.STV_DEV_BAD_SAMPLE),
                                      ("above", stv.STV_DEV_BAD_SAMPLE), ("empty", stv.STV_DEV_BAD_SAMPLE),
                                      ("u", stv.STV_DEV_BAD_SAMPLE), ("u nan", stv.STV_DEV_BAD_SAMPLE),
                                      ("heavy", 0), ("heavy leaf", stv.STV_DEV_BAD_SAMPLE), ("q nan", stv.STV_DEV_BAD_SAMPLE),
                                      ("parent", stv.STV_DEV_BAD_TREE), ("root", stv.STV_DEV_BAD_TREE)])
def test_bad_sequences_alone_are_refused(gpu, what, bit):
    rng = np.random.default_rng(7)
    n, t, vocab = 3, 4, 9000
    p = rows(rng, n * t, vocab, torch.float32, vocab, 1.0).contiguous()
    q = rows(rng, n * t, vocab, torch.float32, vocab, 1.0).contiguous()
    parent = np.tile(tree(rng, t, "star"), (n, 1))
    ids = np.tile(np.array([0, 5, 6, 7]), (n, 1))
    u = np.float32(0.9 + 0.09 * rng.random((n, t)))
    p[:, 5:8] = 0  # every draft is rejected
    want = call(parent, ids, p, q, u)
    r = t  # sequence 1's root row
    if what in ("nan", "negative", "above"):
        p[r, 4321] = {"nan": float("nan"), "negative": -1e-3, "above": 1.5}[what]
    elif what == "empty":
        p[r] = 0
    elif what.startswith("heavy"):  # accepted by the one entry that is read; its own row is added up
        p[r] = 1
        q[r] = 0
        if what == "heavy leaf":
            p[r + 1] = 1
    elif what == "q nan":
        q[r, 77] = float("nan")
    elif what.startswith("u"):
        u[1, 0] = 1.0 if what == "u" else float("nan")
    elif what == "parent":
        parent[1, 2] = 2
    else:
        parent[1, 0] = 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n_commit, path, out = call(parent, ids, p, q, u, status=status)
    assert status.item() == bit
    if bit:
        assert n_commit[1] == 0 and (path[1] == -1).all() and (out[1] == -1).all()
    else:
        assert n_commit[1] == 2 and out[1, 0] == 5 and path[1].tolist() == [0, 1, -1, -1]
    for s in (0, 2):
        assert n_commit[s] == want[0][s] and (out[s] == want[2][s]).all() and (path[s] == want[1][s]).all()


def test_many_sequences_few_tokens_and_graphs(gpu):
    rng = np.random.default_rng(8)
    n, t, vocab = 3000, 3, 5
    p, q = rows(rng, n * t, vocab, torch.float32, vocab, 1.0), rows(rng, n * t, vocab, torch.float32, vocab, 1.0)
    parent, ids = np.tile(tree(rng, t, "chain"), (n, 1)), rng.integers(0, vocab, (n, t))
    u = np.float32(rng.random((n, t)) * 0.9999)
    want = call(parent, ids, p, q, u)
    a = [dev(parent), dev(ids), p, q, dev(u, torch.float32)]
    out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n,), (n, t), (n, t))]
    gr = torch.cuda.CUDAGraph()
    stv.stv_tree_accept_probs(*a, *out)
    with torch.cuda.graph(gr):
        stv.stv_tree_accept_probs(*a, *out)
    for _ in range(2):
        for o in out:
            o.fill_(-5)
        gr.replay()
        assert all(np.array_equal(o.cpu().numpy(), w) for o, w in zip(out, want))
    P, Q = p.double().cpu().numpy(), q.double().cpu().numpy()
    for s in range(0, n, 7):
        path, ids_out, gap = accept(parent[s], ids[s], P[s * t:(s + 1) * t], Q[s * t:(s + 1) * t], u[s].astype(np.float64), False)
        assert gap < 1e-11 or (want[0][s] == len(path) and want[2][s, :len(path)].tolist() == ids_out)
