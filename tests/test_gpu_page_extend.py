"""stv_page_extend against the books in Python, and the page calls on the
drafter's cache."""
import numpy as np
import pytest
import torch

import opkit
import speculative_tree_verify_bit_gb300 as stv
from drafterkit import PAGE, dev

pytestmark = pytest.mark.gpu


def pool_of(b):
    return stv.PagePool(dev(b.refs), dev(b.tables), dev(b.counts))


def extend(pool, seqs, n_new, ctx, max_rows, maps=(True, True, True)):
    n = len(n_new)
    out = [torch.full((max_rows,), -9, dtype=torch.int32, device="cuda") if m else None for m in maps]
    start = torch.full((n + 1,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stv.stv_page_extend(pool, None if seqs is None else dev(seqs), dev(n_new), dev(ctx), start, *out, dev_status=status)
    return start.cpu().numpy(), [None if o is None else o.cpu().numpy() for o in out], status.item()


def want_maps(b, seqs, n_new, max_rows):
    start = np.concatenate([[0], np.cumsum(n_new)])
    maps = np.full((3, max_rows), -1, np.int64)
    for i, (s, k) in enumerate(zip(seqs, n_new)):
        for j in range(k):
            pos = b.ctx[s] + j
            maps[:, start[i] + j] = i, pos, b.tables[s, pos // PAGE] * PAGE + pos % PAGE
    return start, maps


@pytest.mark.parametrize("n,max_ctx,max_new,max_rows", [(1, 0, 1, 1), (1, 255, 2, 5), (3, 600, 0, 4), (40, 900, 3, 200),
                                                        (40, 300, 700, 40 * 700), (200, 60, 5, 4096), (200, 60, 5, 4097)])
@pytest.mark.parametrize("listed", [True, False])
def test_extend(gpu, n, max_ctx, max_new, max_rows, listed):
    rng = np.random.default_rng(n + max_new)
    seqs_all = n + 3
    stride = (max_ctx + max_new) // PAGE + 2
    b = opkit.Books(seqs_all * stride, seqs_all, stride)
    b.ctx[:] = rng.integers(0, max_ctx + 1, seqs_all)
    order = rng.permutation(seqs_all)
    b.reserve(order, 0)
    b.free(order[:2])       # holes in the pool; these two hold nothing, whatever their ctx
    seqs = rng.permutation(seqs_all)[:n] if listed else np.arange(n)
    n_new = rng.integers(0, max_new + 1, n)
    pool = pool_of(b)
    start, maps, status = extend(pool, seqs if listed else None, n_new, b.ctx, max_rows)
    for s, k in zip(seqs, n_new):
        while b.counts[s] * PAGE < b.ctx[s] + k:
            b.take(s)
    assert status == 0
    for got, want in ((pool.refs, b.refs), (pool.tables, b.tables), (pool.counts, b.counts)):
        assert np.array_equal(got.cpu().numpy(), want)
    want_start, want = want_maps(b, seqs, n_new, max_rows)
    assert np.array_equal(start, want_start)
    for got, w in zip(maps, want):
        assert np.array_equal(got, w)
    # nothing to hand out any more: the same maps
    again, maps2, status = extend(pool, seqs if listed else None, n_new, b.ctx, max_rows, (True, False, True))
    assert status == 0 and np.array_equal(again, want_start)
    assert np.array_equal(maps2[0], want[0]) and maps2[1] is None and np.array_equal(maps2[2], want[2])


@pytest.mark.parametrize("seqs,n_new,ctx,rows,bit", [
    ([0, 0], [1, 1], [0, 0, 0], 8, stv.STV_DEV_BAD_SEQ),
    ([0, 3], [1, 1], [0, 0, 0], 8, stv.STV_DEV_BAD_SEQ),
    ([0, -1], [1, 1], [0, 0, 0], 8, stv.STV_DEV_BAD_SEQ),
    ([0, 1], [1, 1], [0, -1, 0], 8, stv.STV_DEV_BAD_SEQ),
    ([0, 1], [1, 1], [0, 3 * PAGE, 0], 8, stv.STV_DEV_BAD_SEQ),          # past the table
    ([0, 1], [1, -1], [0, 0, 0], 8, stv.STV_DEV_BAD_ROW),
    ([0, 1], [5, 4], [0, 0, 0], 8, stv.STV_DEV_BAD_ROW),                 # more rows than there is room for
    ([0, 1], [2**31 - 1, 2**31 - 1], [0, 0, 0], 8, stv.STV_DEV_BAD_ROW | stv.STV_DEV_BAD_SEQ),
    ([0, 1, 2], [600, 600, 600], [0, 0, 0], 5000, stv.STV_DEV_NO_PAGES),
])
def test_extend_is_all_or_nothing(gpu, seqs, n_new, ctx, rows, bit):
    b = opkit.Books(7, 3, 3)
    pool = pool_of(b)
    start, maps, status = extend(pool, seqs, n_new, ctx, rows)
    assert status == bit
    assert (start == 0).all() and all((m == -1).all() for m in maps)
    assert int(pool.refs.sum()) == 0 and int(pool.counts.sum()) == 0 and (pool.tables == -1).all()


def test_extend_on_a_bad_entry(gpu):
    """A sequence that holds a page outside the pool: its rows have no slot."""
    b = opkit.Books(4, 2, 3)
    b.ctx[:] = 250, 10
    b.reserve([0, 1], 0)
    b.tables[1, 0] = 99
    start, maps, status = extend(pool_of(b), [0, 1], [8, 2], b.ctx, 12)
    assert status == stv.STV_DEV_BAD_PAGE and start.tolist() == [0, 8, 10]
    assert maps[2][8:].tolist() == [-1] * 4 and maps[1][8:].tolist() == [10, 11, -1, -1]
    assert maps[2][:8].tolist() == [250, 251, 252, 253, 254, 255, 2 * PAGE, 2 * PAGE + 1]


def test_extend_of_nothing_and_from_a_graph(gpu):
    b = opkit.Books(40, 3, 12)
    pool = pool_of(b)
    start, maps, status = extend(pool, [], [], [0, 0, 0], 5)
    assert status == 0 and start.tolist() == [0] and all((m == -1).all() for m in maps)
    seqs, n_new, ctx = dev([2, 0]), dev([1, 300]), dev([0, 0, 0])
    out = torch.zeros((4, 5000), dtype=torch.int32, device="cuda")
    gr = torch.cuda.CUDAGraph()
    stv.stv_page_extend(pool, seqs, n_new, ctx, out[0, :3], out[1], out[2], out[3])
    with torch.cuda.graph(gr):
        stv.stv_page_extend(pool, seqs, n_new, ctx, out[0, :3], out[1], out[2], out[3])
    b.ctx[:] = 0, 0, 0
    for s, k in ((2, 1), (0, 300)):
        while b.counts[s] * PAGE < k:
            b.take(s)
    for step in range(3):
        ctx += dev([300, 0, 1])
        gr.replay()
        b.ctx += np.array([300, 0, 1], np.int32)
        for s, k in ((2, 1), (0, 300)):
            while b.counts[s] * PAGE < b.ctx[s] + k:
                b.take(s)
        want_start, want = want_maps(b, [2, 0], [1, 300], 5000)
        assert np.array_equal(out[1:].cpu().numpy(), want) and np.array_equal(pool.tables.cpu().numpy(), b.tables)


def test_page_calls_on_the_drafter_cache(gpu):
    """Fork and compact move the row cache's pages as they move the others'."""
    hkv, hd = 2, 64
    shape = stv.make_row_shape(4, hkv, hd, torch.bfloat16)
    assert stv.stv_page_bytes(shape) == hkv * 2 * PAGE * hd * 2
    layers = [stv.RowCache.empty(8, hkv, hd, torch.bfloat16) for _ in range(3)]
    for l in layers:
        l.pool.copy_(torch.randn(l.pool.shape, device="cuda"))
    b = opkit.Books(8, 4, 4)
    b.ctx[:] = 300, 40, 0, 0
    b.reserve([1, 0], 0)
    pool, ctx = pool_of(b), dev(b.ctx)
    before = [l.pool.clone() for l in layers]
    ws = torch.empty(stv.stv_page_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    stv.stv_page_fork(shape, layers, pool, dev([0, 0]), dev([2, 3]), ctx, ws)
    t = pool.tables.cpu().numpy()
    assert t[2, 0] == t[3, 0] == t[0, 0] and len({t[0, 1], t[2, 1], t[3, 1]}) == 3
    for l, old in zip(layers, before):
        for s in (2, 3):
            assert torch.equal(l.pool[int(t[s, 1])], old[int(t[0, 1])])
    stv.stv_page_free(pool, dev([1, 0]))
    page_map, n_live = dev(np.zeros(8)), dev([0])
    stv.stv_page_compact(shape, layers, pool, page_map, n_live, ws)
    t2 = pool.tables.cpu().numpy()
    assert n_live.item() == 3 and t2.max() == 2
    for l, old in zip(layers, before):
        for s in (2, 3):
            assert torch.equal(l.pool[int(t2[s, 0])], old[int(t[0, 0])]) and torch.equal(l.pool[int(t2[s, 1])], old[int(t[0, 1])])
