"""A drafter's life around a verify round, as it would be used: prompts of
unequal lengths get pages and slots, their rows are turned, written and attended
to; then block after block is drafted (rows that see one another), sampled and
verified, the accepted rows' pages kept; a fork goes on alone.  Every attention
output is compared with the 64-bit form over rows kept apart, and the target's
3-bit cache is appended to with the same call's maps."""
import numpy as np
import pytest
import torch

import oracle
import speculative_tree_verify_bit_gb300 as stv
from drafterkit import PAGE, accept, dev, visible

pytestmark = pytest.mark.gpu

HQ, HKV, HD, VOCAB, T, LAYERS = 8, 2, 128, 4099, 6, 2
WINDOW, SINKS = 300, 4
BF16 = torch.bfloat16


class Side:
    """The drafter: weights, caches, books, and every row it ever wrote, apart from the cache."""

    def __init__(self, n_pages, max_seqs, stride):
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.emb, self.w = r(VOCAB, 64), [r(64, (HQ + 2 * HKV) * HD) / 8 for _ in range(LAYERS)]
        self.shape = stv.make_row_shape(HQ, HKV, HD, BF16)
        self.layers = [stv.RowCache.empty(n_pages, HKV, HD, BF16) for _ in range(LAYERS)]
        for l in self.layers:
            l.pool.fill_(float("nan"))
        self.pool = stv.PagePool.empty(n_pages, max_seqs, stride)
        self.ctx = dev(np.zeros(max_seqs))
        self.rope = stv.make_rope(HD, (HD // 2,))
        self.kept = [[{} for _ in range(max_seqs)] for _ in range(LAYERS)]  # position -> (k, v)
        self.status = dev([0])

    def step(self, seqs, tokens, causal):
        """New tokens (a list per sequence) through every layer; checks each layer's output."""
        n_new = [len(t) for t in tokens]
        n, most = sum(n_new), max(n_new)
        start, maps = dev(np.zeros(len(seqs) + 1)), dev(np.zeros((3, n + 5)))
        stv.stv_page_extend(self.pool, dev(seqs), dev(n_new), self.ctx, start, *maps, dev_status=self.status)
        ids = torch.as_tensor(np.concatenate(tokens), device="cuda")
        pos = maps[1].clamp(min=0)[None].contiguous()
        spec = stv.make_attn(WINDOW, SINKS, causal)
        ws = torch.empty(stv.stv_paged_attn_workspace_bytes(self.shape, most), dtype=torch.uint8, device="cuda")
        ctx = self.ctx.tolist()
        for l in range(LAYERS):
            row = torch.zeros((n + 5, HQ + 2 * HKV, HD), dtype=BF16, device="cuda")
            row[:n] = (self.emb[ids] @ self.w[l]).to(BF16).view(n, -1, HD)
            q, k, v = row[:, :HQ], row[:, HQ:HQ + HKV], row[:, HQ + HKV:]
            stv.stv_rope(self.rope, pos, q, q, k, k)
            stv.stv_kv_write(self.shape, self.layers[l], k, v, maps[2], dev_status=self.status)
            o = torch.full((n + 5, HQ, HD), 7.0, dtype=BF16, device="cuda")
            stv.stv_paged_attn(self.shape, spec, self.layers[l], self.pool, dev(seqs), self.ctx, start, most, q, o, ws,
                               dev_status=self.status)
            at = 0
            for s, m in zip(seqs, n_new):
                for j in range(m):
                    self.kept[l][s][ctx[s] + j] = (k[at + j].double(), v[at + j].double())
                self.check(l, s, ctx[s], q[at:at + m].double(), o[at:at + m].double(), causal)
                at += m
            assert (o[n:] == 7.0).all()
        assert self.status.item() == 0
        return start, maps

    def check(self, l, s, ctx, q, o, causal):
        end = ctx + q.shape[0]
        k, v = (torch.stack([self.kept[l][s][i][w] for i in range(end)]) for w in range(2))
        see = visible(np.arange(ctx, end), end, WINDOW, SINKS, causal)
        for h in range(HQ):
            w = torch.softmax((q[:, h] @ k[:, h * HKV // HQ].T * HD ** -0.5).masked_fill(~see, -float("inf")), 1)
            vv = v[:, h * HKV // HQ]
            # three bf16 roundings (P, in its sum too, and the result) and fp32 sums
            half = 2.0 ** -8
            assert ((o[:, h] - w @ vv).abs() <= (w @ vv.abs()) * (3 * half + 2.0 ** -11)).all()


def test_prompts_blocks_verification_and_a_fork(gpu):
    rng = np.random.default_rng(2)
    side = Side(40, 4, 8)
    target_shape = stv.make_shape(24, 4)
    target = stv.LayerCache.empty(40, 4)
    prompts = [rng.integers(0, VOCAB, n) for n in (700, 3, 251)]
    lens = np.array([len(p) for p in prompts])
    seqs = [2, 0, 1]
    start, maps = side.step(seqs, prompts, True)
    # the target's own cache, appended to with the same maps
    n = int(lens.sum())
    k, v = (torch.randn((n, 4, 256), device="cuda").half() for _ in range(2))
    listed = [side.pool.seq(s, -(-int(m) // PAGE), 0) for s, m in zip(seqs, lens)]
    stv.stv_kv_append_pack(target_shape, target, listed, k, v, maps[0, :n].contiguous(), maps[1, :n].contiguous())
    cache = oracle.Cache(4, 40)
    tables = [side.pool.tables[s].cpu().numpy() for s in seqs]
    oracle.kv_append(cache, tables, k.cpu().numpy(), v.cpu().numpy(), maps[0, :n].cpu().numpy(), maps[1, :n].cpu().numpy())
    assert np.array_equal(target.pool.cpu().numpy(), cache.pool)
    for s, m in zip(seqs, lens):
        side.ctx[s] = int(m)

    parent = np.tile(np.arange(-1, T - 1), (3, 1))
    for step in range(4):
        # a block of drafts (they see one another), or one token
        drafts = rng.integers(0, VOCAB, (3, T))
        if step == 2:
            side.step(seqs, [d[:1] for d in drafts], True)
            side.ctx += dev([1, 1, 1, 0])
            continue
        side.step(seqs, list(drafts), False)
        p, q = (torch.softmax(torch.randn((3 * T, VOCAB), device="cuda") * 2, 1) for _ in range(2))
        for s in range(3):  # likely drafts, so that some are accepted
            for i in range(1, T):
                p[s * T + i - 1, drafts[s, i]] += 1.0
                q[s * T + i - 1, drafts[s, i]] += 0.5 * (1 + step)
        p, q = p / p.sum(1, keepdim=True), q / q.sum(1, keepdim=True)
        u = torch.rand((3, T), device="cuda")
        nc, path, out = dev(np.zeros(3)), dev(np.zeros((3, T))), dev(np.zeros((3, T)))
        stv.stv_tree_accept_probs(dev(parent), dev(drafts), p, q, u, nc, path, out, dev_status=side.status)
        for i in range(3):
            want = accept(parent[i], drafts[i], p[i * T:(i + 1) * T].double().cpu().numpy(),
                          q[i * T:(i + 1) * T].double().cpu().numpy(), u[i].double().cpu().numpy(), False)
            m = int(nc[i])
            assert path[i, :m].tolist() == want[0] and out[i, :m].tolist() == want[1]
            # a chain's accepted rows stay where they are; the rows after them are written again
            side.ctx[seqs[i]] += m
    assert side.status.item() == 0

    # a sample of sequence 2 goes on by itself
    ws = torch.empty(stv.stv_page_workspace_bytes(side.pool), dtype=torch.uint8, device="cuda")
    stv.stv_page_fork(side.shape, side.layers, side.pool, dev([2]), dev([3]), side.ctx, ws, dev_status=side.status)
    for l in range(LAYERS):
        side.kept[l][3] = dict(side.kept[l][2])
    side.step([3, 2], [rng.integers(0, VOCAB, 200), rng.integers(0, VOCAB, 2)], True)
    assert side.pool.tables[3, 0] == side.pool.tables[2, 0] and side.status.item() == 0
