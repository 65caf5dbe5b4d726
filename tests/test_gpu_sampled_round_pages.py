"""What the rounds of forked samples write.  The prompt ends three tokens
before a page does, so the page that the fork copies fills within the rounds
and the rows after it go to a page that reserve handed out; every committed
token's K and V, in those pages too, must be what the same rounds write into
pages of each sample's own, before a compaction and after it.  (Both sides run
the same sequences in a call: the split plan, and so the attention's rounding,
is the batch's.)"""
import numpy as np
import pytest
import torch

import oracle
import speculative_tree_verify_bit_gb300 as stv
import workloads
from test_gpu_sampled_round import HKV, HQ, LAYERS, RD, SEC, T, VOCAB, Model, one_round

pytestmark = pytest.mark.gpu

PROMPT, SAMPLES, SEQS, STRIDE, PAGES = 765, 3, 5, 6, 26


def dev(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


def prefill(model, spec, layers, seq):
    ids = np.random.default_rng(40).integers(0, VOCAB, PROMPT)
    pos = torch.arange(PROMPT, dtype=torch.int32, device="cuda").expand(3, PROMPT).contiguous()
    for l, layer in enumerate(layers):
        _, k, v = model.rows(ids, l)
        kr = torch.empty_like(k, memory_format=torch.contiguous_format)
        stv.stv_rope(spec, pos, None, None, k, kr)
        stv.stv_kv_append_pack(model.shape, layer, [seq], kr, v.contiguous(), torch.zeros_like(pos[0]), pos[0])


def decoded(layer, table, begin, end):
    cache = oracle.Cache(HKV, layer.n_pages, layer.pool.cpu().numpy())
    return [oracle.decode(cache, [table], 0, begin, end, which) for which in ("k", "v")]


def test_rounds_write_what_they_write_alone(gpu):
    model, spec = Model(), stv.make_rope(RD, SEC, theta=1e6)
    model.shape = shape = stv.make_shape(HQ, HKV)
    rng = np.random.default_rng(41)
    pool = stv.PagePool.empty(PAGES, SEQS, STRIDE)
    layers = [stv.LayerCache.empty(PAGES, HKV) for _ in range(LAYERS)]
    ctx = dev([0, 900, 0, 0, PROMPT])
    ws = torch.empty(stv.stv_page_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stv.stv_page_reserve(pool, dev([1, 4]), ctx, 0, dev_status=status)
    stv.stv_page_free(pool, dev([1]), dev_status=status)
    prefill(model, spec, layers, pool.seq(4, 3, 0))
    stv.stv_page_fork(shape, layers, pool, dev([4] * SAMPLES), dev([0, 1, 2]), ctx, ws, dev_status=status)
    first = pool.tables[:, :3].tolist()
    assert all(first[s][:2] == first[4][:2] and first[s][2] != first[4][2] for s in range(SAMPLES))

    own = [stv.LayerCache.empty(SAMPLES * STRIDE, HKV) for _ in range(LAYERS)]
    table = torch.arange(SAMPLES * STRIDE, dtype=torch.int32, device="cuda").view(SAMPLES, STRIDE)
    for s in range(SAMPLES):
        prefill(model, spec, own, stv.Seq(table[s], 0))
    at = [PROMPT] * SAMPLES
    live = [0, 1, 2]

    def compare():
        own_pages = reserved = 0
        for s in live:
            mine = pool.tables[s].tolist()
            assert int(ctx[s].item()) == at[s]
            for l in range(LAYERS):
                a, b = layers[l].pool.view(PAGES, -1), own[l].pool.view(SAMPLES * STRIDE, -1)
                for e in range(at[s] // 256):
                    assert torch.equal(a[mine[e]], b[s * STRIDE + e])
                    own_pages += e >= 2
                held = -(-at[s] // 256)
                for got, want in zip(decoded(layers[l], mine[:held], 512, at[s]),
                                     decoded(own[l], table[s].tolist(), 512, at[s])):
                    assert np.array_equal(got, want) and np.abs(want).max(axis=(1, 2)).min() > 0
                reserved += at[s] > 768
        return own_pages, reserved

    page_map, n_live = torch.empty(PAGES, dtype=torch.int32, device="cuda"), dev([0])
    for rnd in range(5):
        tokens = [rng.integers(0, VOCAB, T) for _ in range(SAMPLES)]
        parents = [workloads.random_tree(rng, T, 4) for _ in range(SAMPLES)]
        u = torch.as_tensor(rng.random((SAMPLES, T)).astype(np.float32), device="cuda").clamp_(max=0.999999)
        stv.stv_page_reserve(pool, dev(live), ctx, T, dev_status=status)
        seqs = [pool.seq(s, -(-(at[s] + T) // 256), at[s]) for s in live]
        rows = torch.as_tensor(live, device="cuda")
        round_ctx = ctx[rows].contiguous()
        rest = [tokens[s] for s in live], [parents[s] for s in live], u[live].reshape(-1).contiguous()
        got = one_round(model, shape, spec, layers, seqs, round_ctx, *rest)
        ctx[rows] = round_ctx
        alone = one_round(model, shape, spec, own, [stv.Seq(table[s], at[s]) for s in live], None, *rest)
        assert got == alone
        for s, ids in zip(live, got):
            at[s] += len(ids)
        compare()
        if rnd == 2:  # holes for the compaction, some of them under pages of the samples that go on
            stv.stv_page_free(pool, dev([4, live.pop(0)]), dev_status=status)
            before = pool.tables.tolist()
            stv.stv_page_compact(shape, layers, pool, page_map, n_live, ws, dev_status=status)
            assert any(pool.tables[s, 2:4].tolist() != before[s][2:4] for s in live)
            compare()
    own_pages, reserved = compare()
    assert own_pages == reserved == len(live) * LAYERS  # full copied pages, and rows in reserved ones
    assert int(status.item()) == 0
