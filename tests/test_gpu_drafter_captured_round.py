"""A drafter's rounds on the GPU alone: pages and slots for the tokens that
the last round committed (as many as they were, in maps of a fixed size), their
rows turned, written and attended to, drafts sampled one by one, and accepted
against the target's probabilities; what is committed is the next round's input.
Captured once and replayed, next to the same rounds run eagerly."""
import numpy as np
import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from drafterkit import PAGE, Drafter, accept, attention, dev

pytestmark = pytest.mark.gpu

HQ, HKV, HD, VOCAB, T, N, ROWS, MOST = 8, 2, 64, 500, 6, 3, 70, 24
PROMPTS = [17, 1, 24]
WINDOW, SINKS = 40, 3
BF16 = torch.bfloat16


class Rounds:
    def __init__(self):
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.emb, self.w = r(VOCAB, 32), r(32, (HQ + 2 * HKV) * HD) / 6
        self.head, self.target = r(T, HQ * HD, VOCAB) / 8, r(VOCAB, VOCAB)
        # (one object for the 64-bit form, which looks at its books and data)
        self.d = Drafter([], HKV, HD, BF16, n_pages=9, max_seqs=4)
        self.d.pool = self.pool = stv.PagePool.empty(9, 4, 3)
        self.shape, self.spec = stv.make_row_shape(HQ, HKV, HD, BF16), stv.make_attn(WINDOW, SINKS)
        self.rope = stv.make_rope(HD, (HD // 2,))
        self.ws = torch.empty(stv.stv_paged_attn_workspace_bytes(self.shape, MOST), dtype=torch.uint8, device="cuda")
        self.seqs, self.parent = dev([2, 0, 3]), dev(np.tile(np.arange(-1, T - 1), (N, 1)))
        self.ctx, self.start, self.status = dev([0] * 4), dev([0] * (N + 1)), dev([0])
        self.ctx[self.seqs.long()] = dev([PAGE - 9, 300, 0])  # as if they had been there before
        self.before = self.ctx.clone()
        stv.stv_page_reserve(self.pool, self.seqs, self.ctx, 0)
        self.d.data.copy_(r(*self.d.data.shape))
        self.row_seq, self.row_pos, self.slots = (dev([0] * ROWS) for _ in range(3))
        self.n_new, self.tokens = dev(PROMPTS), torch.randint(0, VOCAB, (N, MOST), generator=g, device="cuda")
        self.o = torch.zeros((ROWS, HQ, HD), dtype=BF16, device="cuda")
        self.drafts, self.u, self.u_drafts = dev(np.zeros((N, T))), r(N, T), r(N * T)
        self.nc, self.path, self.out = dev([0] * N), dev(np.zeros((N, T))), dev(np.zeros((N, T)))
        self.p = self.q = None

    def step(self):
        stv.stv_page_extend(self.pool, self.seqs, self.n_new, self.ctx, self.start, self.row_seq, self.row_pos, self.slots,
                            dev_status=self.status)
        at = self.row_seq.clamp(min=0).long()
        first = self.ctx[self.seqs.long()]
        ids = self.tokens[at, (self.row_pos - first[at]).clamp(min=0).long()]
        self.row = (self.emb[ids] @ self.w).to(BF16).view(ROWS, HQ + 2 * HKV, HD)
        qr, k, v = self.row[:, :HQ], self.row[:, HQ:HQ + HKV], self.row[:, HQ + HKV:]
        stv.stv_rope(self.rope, self.row_pos.clamp(min=0)[None].contiguous(), qr, qr, k, k)
        stv.stv_kv_write(self.shape, stv.RowCache(self.d.data), k, v, self.slots, dev_status=self.status)
        stv.stv_paged_attn(self.shape, self.spec, stv.RowCache(self.d.data), self.pool, self.seqs, self.ctx, self.start, MOST, qr,
                           self.o, self.ws, dev_status=self.status)
        # drafts from the last row's output, one head each; node i's children are drawn from row i
        last = self.o[(self.start[1:] - 1).long()].float().flatten(1)
        logits = torch.einsum("nd,tdv->ntv", last, self.head).flatten(0, 1).contiguous()
        drawn = torch.empty(N * T, dtype=torch.int32, device="cuda")
        stv.stv_sample(logits, self.u_drafts, drawn, dev_status=self.status)
        self.drafts[:, 1:] = drawn.view(N, T)[:, :-1]
        final = self.tokens[torch.arange(N, device="cuda"), (self.n_new - 1).long()]
        nodes = torch.cat([final[:, None], self.drafts[:, 1:].long()], 1)
        self.q = torch.softmax(logits, 1)
        self.p = torch.softmax(logits + 0.7 * self.target[nodes].flatten(0, 1), 1)
        stv.stv_tree_accept_probs(self.parent, self.drafts, self.p, self.q, self.u, self.nc, self.path, self.out,
                                  dev_status=self.status)
        self.ctx.index_add_(0, self.seqs.long(), self.n_new)
        self.n_new.copy_(self.nc)
        self.tokens[:, :T] = self.out.clamp(min=0)

    def state(self):
        return [self.pool.refs, self.pool.tables, self.pool.counts, self.d.data, self.ctx, self.start, self.row_seq, self.row_pos,
                self.slots, self.n_new, self.tokens, self.o, self.drafts, self.nc, self.path, self.out]


def test_captured_rounds_are_the_eager_ones(gpu):
    rng = np.random.default_rng(3)
    eager, captured = Rounds(), Rounds()
    start = [t.clone() for t in captured.state()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    captured.u.fill_(0.5)
    captured.u_drafts.fill_(0.5)
    with torch.cuda.stream(side):
        captured.step()  # (the libraries' first calls are not captured)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for t, was in zip(captured.state(), start):
        t.copy_(was)
    lengths = set()
    for step in range(12):
        u = torch.as_tensor(rng.random((2, N, T)) * 0.999, dtype=torch.float32, device="cuda")
        for r in (eager, captured):
            r.u.copy_(u[0])
            r.u_drafts.copy_(u[1].flatten())
        n_new, ctx = eager.n_new.tolist(), eager.ctx.tolist()
        eager.step()
        graph.replay()
        for a, b in zip(eager.state(), captured.state()):
            assert torch.equal(a, b)
        assert eager.status.item() == 0 and captured.status.item() == 0
        assert eager.start.tolist() == [0] + np.cumsum(n_new).tolist()
        # the 64-bit forms: attention, and acceptance
        rows = sum(n_new)
        entries = [(s, ctx[s], eager.start.tolist()[i], n) for i, (s, n) in enumerate(zip([2, 0, 3], n_new))]
        want, tol = attention(eager.d, eager.row[:, :HQ], entries, window=WINDOW, sinks=SINKS)
        assert ((eager.o.double() - want).abs() <= tol)[:rows].all()
        assert (eager.row_seq[rows:] == -1).all() and (eager.slots[rows:] == -1).all()
        P, Q = eager.p.double().cpu().numpy().reshape(N, T, -1), eager.q.double().cpu().numpy().reshape(N, T, -1)
        for i in range(N):
            path, out, gap = accept(eager.parent[i].tolist(), eager.drafts[i].tolist(), P[i], Q[i],
                                    u[0, i].double().cpu().numpy(), False)
            m = len(path)
            lengths.add(m)
            assert gap < 1e-11 or (eager.nc[i].item() == m and eager.out[i, :m].tolist() == out)
    assert len(lengths) > 2  # some drafts were accepted, some not
    assert all(int(eager.ctx[s]) > int(eager.before[s]) + 24 for s in (2, 0, 3))
