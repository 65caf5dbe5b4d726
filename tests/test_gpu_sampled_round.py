"""The operators around a round, run as a serving loop uses them: one prompt's
cache forked for several samples, their pages reserved, the tree's q and k
rows turned to their positions, appended, verified and merged, the target's
tokens drawn, the trees accepted and committed, samples freed and the pool
compacted -- against the same rounds on caches of their own, built without
forks, page pools or compaction."""
import numpy as np
import pytest
import torch

import opkit
import oracle
import speculative_tree_verify_bit_gb300 as stv
import workloads

pytestmark = pytest.mark.gpu

T, HQ, HKV, LAYERS, VOCAB, RD, SEC = 8, 24, 4, 2, 5003, 64, (12, 10, 10)


class Model:
    """Stands in for the target: q, k, v rows of a token at a layer and the
    logits of a node are draws seeded by what they depend on."""

    def rows(self, tokens, layer):
        g = torch.Generator(device="cuda")
        out = []
        for t in tokens:
            g.manual_seed(int(t) * 64 + layer)
            out.append(torch.randn((HQ + 2 * HKV, 256), generator=g, device="cuda").half())
        x = torch.stack(out)
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def logits(self, o):
        """From the last layer's output: any deterministic function of it."""
        w = torch.Generator(device="cuda").manual_seed(5)
        m = torch.randn((256, VOCAB), generator=w, device="cuda")
        return ((o.float().mean(1) @ m) * 8).bfloat16()


def positions(ctx, parent):
    depth = np.zeros(len(parent), np.int64)
    for i in range(1, len(parent)):
        depth[i] = depth[parent[i]] + 1
    return np.tile(ctx + depth, (3, 1)).astype(np.int32)


def one_round(model, shape, spec, layers, seqs, ctx_dev, tokens, parents, u):
    """tokens, parents [n][T]; returns the committed ids per sequence."""
    n = len(seqs)
    dev = lambda a: torch.as_tensor(a, device="cuda")
    pos = dev(np.concatenate([positions(s.ctx, p) for s, p in zip(seqs, parents)], 1))
    par = dev(np.stack(parents).astype(np.int32))
    row_seq = dev(np.repeat(np.arange(n, dtype=np.int32), T))
    row_pos = dev(np.concatenate([s.ctx + np.arange(T) for s in seqs]).astype(np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.empty((n, T, HQ, 256), dtype=torch.float16, device="cuda")
    ws = torch.empty(stv.stv_verify_workspace_bytes(shape, seqs, T), dtype=torch.uint8, device="cuda")
    for l, layer in enumerate(layers):
        q, k, v = model.rows(np.concatenate(tokens), l)
        qr, kr = torch.empty((n * T, HQ, 256), dtype=torch.float16, device="cuda"), torch.empty(
            (n * T, HKV, 256), dtype=torch.float16, device="cuda")
        stv.stv_rope(spec, pos, q, qr, k, kr)
        stv.stv_kv_append_pack(shape, layer, seqs, kr, v.contiguous(), row_seq, row_pos, dev_status=status)
        stv.stv_verify_attn(shape, layer, seqs, qr.view(n, T, HQ, 256), par, T, "exact", ws, dev_status=status)
        stv.stv_split_combine(shape, seqs, T, ws, o)
    ids = torch.empty(n * T, dtype=torch.int32, device="cuda")
    logits = model.logits(o.view(n * T, HQ, 256))
    stv.stv_sample(logits, u, ids, temperature=torch.full((n,), 0.9, device="cuda"),
                   top_p=torch.full((n,), 0.95, device="cuda"), rows_per_param=T, dev_status=status)
    nc = torch.zeros(n, dtype=torch.int32, device="cuda")
    path = torch.zeros((n, T), dtype=torch.int32, device="cuda")
    out = torch.zeros((n, T), dtype=torch.int32, device="cuda")
    drafts = dev(np.stack(tokens).astype(np.int32))
    target = ids.view(n, T)
    # half of the drafts are what the target drew at their parent, so that paths are accepted
    for s in range(n):
        for c in range(1, T, 2):
            drafts[s, c] = target[s, int(parents[s][c])]
    stv.stv_tree_accept(par, drafts, target, nc, path, out, dev_status=status)
    stv.stv_kv_commit(shape, layers, seqs, T, nc, path, ctx_dev=ctx_dev, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # the draw and the acceptance against their plain forms
    x, uu = logits.double().cpu().numpy(), u.cpu().numpy()
    for r in range(n * T):
        want, _, gap = opkit.sample(x[r], uu[r], 0.9, 0, 0.95)
        assert gap <= 2.0 ** -28 or int(ids[r]) == want
    got = []
    for s in range(n):
        c = int(nc[s].item())
        w_n, w_path, w_ids = oracle.tree_accept(parents[s], drafts[s].cpu().numpy(), target[s].cpu().numpy())
        assert c == w_n and path[s, :c].tolist() == w_path.tolist() and out[s, :c].tolist() == w_ids.tolist()
        got.append(out[s, :c].tolist())
    return got


def test_forked_samples_equal_samples_of_their_own(gpu):
    model, spec, shape = Model(), stv.make_rope(RD, SEC, theta=1e6), stv.make_shape(HQ, HKV)
    prompt, samples, max_seqs, stride, n_pages = 600, 3, 5, 6, 24
    rng = np.random.default_rng(4)
    prompt_ids = rng.integers(0, VOCAB, prompt)
    dev = lambda a: torch.as_tensor(np.asarray(a, np.int32), device="cuda")

    def prefill(layers, seq):
        pos = torch.arange(prompt, dtype=torch.int32, device="cuda").expand(3, prompt).contiguous()
        for l, layer in enumerate(layers):
            _, k, v = model.rows(prompt_ids, l)
            kr = torch.empty_like(k, memory_format=torch.contiguous_format)
            stv.stv_rope(spec, pos, None, None, k, kr)
            stv.stv_kv_append_pack(shape, layer, [seq], kr, v.contiguous(), torch.zeros_like(pos[0]), pos[0])

    # the pool: sequence 4 holds the prompt (pages taken after a sequence that is freed again: holes)
    pool = stv.PagePool.empty(n_pages, max_seqs, stride)
    layers = [stv.LayerCache.empty(n_pages, HKV) for _ in range(LAYERS)]
    ctx = dev([0, 900, 0, 0, prompt])
    ws = torch.empty(stv.stv_page_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stv.stv_page_reserve(pool, dev([1, 4]), ctx, 0, dev_status=status)
    stv.stv_page_free(pool, dev([1]), dev_status=status)
    prefill(layers, pool.seq(4, 3, 0))
    stv.stv_page_fork(shape, layers, pool, dev([4] * samples), dev([0, 1, 2]), ctx, ws, dev_status=status)

    # each sample alone: its own pool, the prompt appended again
    alone = []
    for _ in range(samples):
        own = [stv.LayerCache.empty(stride, HKV) for _ in range(LAYERS)]
        table = torch.arange(stride, dtype=torch.int32, device="cuda")
        prefill(own, stv.Seq(table, 0))
        alone.append([own, table, prompt])

    live, out_a, out_b = [0, 1, 2], {s: [] for s in range(samples)}, {s: [] for s in range(samples)}
    host_ctx = {s: prompt for s in live}
    page_map, n_live = torch.empty(n_pages, dtype=torch.int32, device="cuda"), dev([0])
    for rnd in range(4):
        tokens = [rng.integers(0, VOCAB, T) for _ in range(samples)]
        parents = [workloads.random_tree(rng, T, 4) for _ in range(samples)]
        u = torch.as_tensor(rng.random((samples, T)).astype(np.float32), device="cuda")
        u.clamp_(max=0.999999)
        stv.stv_page_reserve(pool, dev(live), ctx, T, dev_status=status)
        seqs = [pool.seq(s, -(-(host_ctx[s] + T) // 256), host_ctx[s]) for s in live]
        # the round's ctx_dev has one entry per sequence of the round
        round_ctx = ctx[torch.as_tensor(live, device="cuda")].contiguous()
        got = one_round(model, shape, spec, layers, seqs, round_ctx, [tokens[s] for s in live],
                        [parents[s] for s in live], u[live].reshape(-1).contiguous())
        ctx[torch.as_tensor(live, device="cuda")] = round_ctx
        for s, ids in zip(live, got):
            out_a[s].append(ids)
            host_ctx[s] += len(ids)
        for s in live:
            own, table, c = alone[s]
            one = one_round(model, shape, spec, own, [stv.Seq(table, c)], None, [tokens[s]], [parents[s]],
                            u[s].contiguous())
            out_b[s].append(one[0])
            alone[s][2] += len(one[0])
        # the cached rows of both are the same bytes, page by page up to the context
        for s in live:
            own, table, c = alone[s]
            assert c == host_ctx[s] == int(ctx[s].item())
            mine = pool.tables[s].tolist()
            for l in range(LAYERS):
                a = layers[l].pool.view(n_pages, -1)
                b = own[l].pool.view(stride, -1)
                for e in range(c // 256):
                    assert torch.equal(a[mine[e]], b[e])
        if rnd == 1:  # one sample ends, and the prompt's own sequence
            stv.stv_page_free(pool, dev([4, live.pop(1)]), dev_status=status)
        if rnd == 2:
            stv.stv_page_compact(shape, layers, pool, page_map, n_live, ws, dev_status=status)
            held = sorted(set(pool.tables[pool.tables >= 0].tolist()))
            assert held == list(range(int(n_live.item())))
    assert out_a == out_b
    assert any(len(ids) > 1 for s in out_a for ids in out_a[s])
    stv.stv_page_free(pool, dev(live), dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and not pool.refs.any()
