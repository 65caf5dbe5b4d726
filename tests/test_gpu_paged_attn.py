"""stv_kv_write and stv_paged_attn against 64-bit forms, at the sizes, masks
and strides where they can go wrong."""
import numpy as np
import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from drafterkit import PAGE, Drafter, attention, dev

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16


def call(d, q, entries, max_new=None, window=0, sinks=0, causal=True, scale=0.0, o=None, status=None, use_seqs=True,
         ws=None):
    """entries: (sequence, ctx, first row, rows), rows in order."""
    n, hq = len(entries), q.shape[1]
    shape = stv.make_row_shape(hq, d.hkv, d.hd, d.dtype)
    max_new = max_new or max([e[3] for e in entries] + [1])
    ctx = np.zeros(d.pool.counts.numel(), np.int64)
    for s, c, _, _ in entries:
        ctx[s] = c
    start = [entries[0][2]] + [e[2] + e[3] for e in entries]
    if ws is None:
        ws = torch.full((stv.stv_paged_attn_workspace_bytes(shape, max_new),), 0xff, dtype=torch.uint8, device="cuda")
    o = torch.full_like(q, 7.0, memory_format=torch.contiguous_format) if o is None else o
    spec = stv.make_attn(window, sinks, causal, scale)
    stv.stv_paged_attn(shape, spec, d.layer, d.pool, dev([e[0] for e in entries]) if use_seqs else None, dev(ctx),
                       dev(start), max_new, q, o, ws, dev_status=status)
    return o


def check(d, q, entries, got, **kw):
    want, tol = attention(d, q, entries, **kw)
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for _, _, row, n in entries:
        inside[row:row + n] = True
    err = (got.double() - want).abs()
    bad = (err > tol) | err.isnan()
    assert not bad[inside].any(), (float((err / tol)[inside].max()), int(bad[inside].sum()))
    assert (got[~inside] == 7.0).all()


def ragged(lens_new, order=None):
    """Entries for (ctx, rows) per sequence, rows one after the other."""
    out, row = [], 0
    for s, (c, n) in enumerate(lens_new):
        out.append((s, c, row, n))
        row += n
    return out, row


MASKS = [dict(), dict(window=1), dict(window=5, sinks=1), dict(window=64), dict(window=100, sinks=4),
         dict(window=200, sinks=70), dict(window=3000, sinks=300), dict(causal=False), dict(causal=False, window=33, sinks=65)]
TOKENS = [(0, 1), (1, 1), (62, 1), (63, 1), (64, 1), (100, 1), (254, 1), (255, 1), (256, 1), (700, 1), (1500, 1)]


@pytest.mark.parametrize("mask", MASKS, ids=str)
@pytest.mark.parametrize("hkv,g,hd,dtype", [(4, 6, 256, FP16), (2, 16, 128, BF16), (1, 1, 64, BF16), (8, 3, 64, FP16)])
def test_single_tokens(gpu, hkv, g, hd, dtype, mask):
    entries, n = ragged(TOKENS)
    d = Drafter([c + k for c, k in TOKENS], hkv, hd, dtype, seed=hd + g)
    q = d.rows(n, hkv * g)
    check(d, q, entries, call(d, q, entries, **mask), **mask)


@pytest.mark.parametrize("mask", MASKS, ids=str)
@pytest.mark.parametrize("hkv,g,hd,dtype", [(2, 6, 256, BF16), (2, 4, 128, FP16), (1, 24, 128, BF16), (2, 7, 64, FP16),
                                            (1, 128, 64, BF16), (3, 1, 256, FP16)])
def test_blocks(gpu, hkv, g, hd, dtype, mask):
    """Ragged blocks, one with no rows among them; more rows than one row tile holds."""
    lens = [(0, 17), (5, 0), (47, 17), (255, 2), (300, 9), (63, 1), (900, 16)]
    entries, n = ragged(lens)
    d = Drafter([c + k for c, k in lens], hkv, hd, dtype, seed=hd + g)
    q = d.rows(n + 3, hkv * g)
    check(d, q, entries, call(d, q, entries, **mask), **mask)


@pytest.mark.parametrize("mask", [dict(), dict(window=130, sinks=3), dict(window=64, sinks=200), dict(causal=False)], ids=str)
@pytest.mark.parametrize("hkv,g,hd,dtype", [(1, 6, 256, FP16), (2, 3, 128, BF16), (1, 2, 64, FP16)])
def test_prompts(gpu, hkv, g, hd, dtype, mask):
    lens = [(0, 321), (100, 1), (257, 640), (0, 127)]
    entries, n = ragged(lens)
    d = Drafter([c + k for c, k in lens], hkv, hd, dtype, seed=hd)
    q = d.rows(n, hkv * g)
    check(d, q, entries, call(d, q, entries, **mask), **mask)


@pytest.mark.parametrize("hd,dtype", [(256, FP16), (128, BF16), (64, FP16)])
def test_long_context_split_over_the_sms(gpu, hd, dtype):
    """One long sequence among short ones: every unit is cut and joined."""
    lens = [(30, 1), (20000, 1), (0, 1)]
    entries, n = ragged(lens)
    d = Drafter([c + k for c, k in lens], 2, hd, dtype, seed=3)
    q = 3 * d.rows(n, 8)
    check(d, q, entries, call(d, q, entries))
    lens = [(9000, 40), (100, 40)]
    entries, n = ragged(lens)
    d = Drafter([c + k for c, k in lens], 1, hd, dtype, seed=4)
    q = 3 * d.rows(n, 4)
    check(d, q, entries, call(d, q, entries))


def test_entries_in_any_order_and_a_first_row(gpu):
    d = Drafter([400, 90, 700], 2, 128, BF16, seed=5)
    entries = [(2, 690, 3, 2), (0, 399, 5, 1), (1, 80, 6, 2)]
    q = d.rows(12, 8)
    check(d, q, entries, call(d, q, entries))
    check(d, q, entries, call(d, q, entries, max_new=50))  # the other kernel


def test_without_row_start(gpu):
    d = Drafter([1, 300, 65], 2, 64, FP16, seed=6)
    q = d.rows(5, 4)
    shape = stv.make_row_shape(4, 2, 64, FP16)
    ws = torch.empty(stv.stv_paged_attn_workspace_bytes(shape, 1), dtype=torch.uint8, device="cuda")
    o = torch.full_like(q, 7.0)
    stv.stv_paged_attn(shape, stv.make_attn(), d.layer, d.pool, dev([0, 1, 2]), dev([0, 299, 64]), None, 1, q, o, ws)
    check(d, q, [(0, 0, 0, 1), (1, 299, 1, 1), (2, 64, 2, 1)], o)


@pytest.mark.parametrize("max_new", [1, 40])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_strided_views(gpu, max_new, pad):
    """q inside a projection's rows, o beside it; strides that allow no 16-byte accesses."""
    d = Drafter([300, 77], 2, 128, BF16, seed=7)
    n = max_new
    entries = [(0, 300 - n, 0, n), (1, 77 - n, n, n)]
    row = torch.zeros((2 * n, 8 * 128 + 8 * 128 + pad), dtype=BF16, device="cuda")
    row[:, :8 * 128] = d.rows(2 * n, 8).flatten(1)
    q, o = row[:, :8 * 128].unflatten(1, (8, 128)), row[:, 8 * 128:16 * 128].unflatten(1, (8, 128))
    if pad:
        row[:, -pad:] = 5.0
    check(d, q, entries, call(d, q, entries, o=o))
    assert pad == 0 or (row[:, -pad:] == 5.0).all()
    # heads further apart, and an address that is no multiple of 16
    flat = torch.zeros(2 * n * 8 * 131 + 1, dtype=BF16, device="cuda")
    q2 = flat[1:].view(2 * n, 8, 131)[:, :, :128]
    q2.copy_(q)
    check(d, q2, entries, call(d, q2, entries))


@pytest.mark.parametrize("n", [1, 30])
def test_what_a_window_leaves_behind_is_not_read(gpu, n):
    """Pages outside window and first tokens have been given up: their table
    entries are -1, and what they held is NaN."""
    d = Drafter([3000], 2, 128, FP16, seed=8)
    q = d.rows(n, 8)
    entries = [(0, 3000 - n, 0, n)]
    mask = dict(window=500, sinks=10)
    want, tol = attention(d, q, entries, **mask)
    for e in range(1, 9):
        d.data[int(d.pool.tables[0, e])] = float("nan")
        d.pool.tables[0, e] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(d, q, entries, status=status, **mask)
    assert ((got.double() - want).abs() <= tol).all() and status.item() == 0


@pytest.mark.parametrize("n", [1, 30])
def test_missing_pages_are_left_out_and_reported(gpu, n):
    d = Drafter([1000, 700], 2, 64, BF16, seed=9)
    q = d.rows(2 * n, 4)
    entries = [(0, 1000 - n, 0, n), (1, 700 - n, n, n)]
    want, tol = attention(d, q, entries)
    part, tol_part = attention(d, q, entries, hidden=(256,))
    keep = d.pool.tables.clone()
    for bad in (-1, 1 << 30):
        d.pool.tables[1, 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = call(d, q, entries, status=status).double()
        assert status.item() == stv.STV_DEV_BAD_PAGE
        assert ((got - want).abs() <= tol)[:n].all() and ((got - part).abs() <= tol_part)[n:].all()
    d.pool.tables.copy_(keep)
    # no pages at all: rows of zeros
    counts = d.pool.counts.clone()
    d.pool.counts[1] = 0
    status.zero_()
    got = call(d, q, entries, status=status).double()
    assert status.item() == stv.STV_DEV_BAD_PAGE and (got[n:] == 0).all() and ((got - want).abs() <= tol)[:n].all()
    d.pool.counts.copy_(counts)


@pytest.mark.parametrize("max_new", [2, 40])
@pytest.mark.parametrize("start,bit", [([0, 1, 9], stv.STV_DEV_BAD_ROW), ([-1, 1, 2], stv.STV_DEV_BAD_ROW),
                                       ([1, 0, 2], stv.STV_DEV_BAD_ROW)])
def test_bad_rows_are_left_out(gpu, max_new, start, bit):
    d = Drafter([400, 200], 2, 64, BF16, seed=10)
    q = d.rows(4, 4)
    shape = stv.make_row_shape(4, 2, 64, BF16)
    ws = torch.empty(stv.stv_paged_attn_workspace_bytes(shape, max_new), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    stv.stv_paged_attn(shape, stv.make_attn(), d.layer, d.pool, None, dev([399, 198]), dev(start), max_new, q, o, ws, status)
    assert status.item() == bit
    entries = [(s, (399, 198)[s], start[s], start[s + 1] - start[s]) for s in range(2)]
    good = [e for e in entries if e[2] >= 0 and e[3] >= 0 and e[2] + e[3] <= 4 and e[3] <= max_new]
    check(d, q, good, o)


@pytest.mark.parametrize("seqs,ctx", [([0, 7], [399, 198]), ([-1, 1], [399, 198]), ([0, 1], [399, -5]),
                                      ([0, 1], [399, (1 << 30) + 1])])
def test_bad_sequences_are_left_out(gpu, seqs, ctx):
    d = Drafter([400, 200], 2, 64, BF16, seed=11)
    q = d.rows(2, 4)
    shape = stv.make_row_shape(4, 2, 64, BF16)
    ws = torch.empty(stv.stv_paged_attn_workspace_bytes(shape, 1), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    stv.stv_paged_attn(shape, stv.make_attn(), d.layer, d.pool, dev(seqs), dev(ctx), None, 1, q, o, ws, status)
    assert status.item() == stv.STV_DEV_BAD_SEQ
    check(d, q, [(s, c, i, 1) for i, (s, c) in enumerate(zip(seqs, ctx)) if 0 <= s < 2 and (s, c) in ((0, 399), (1, 198))], o)


@pytest.mark.parametrize("n", [1, 20])
def test_large_scores_and_a_scale(gpu, n):
    """Scores far apart (one key takes all) and a maximum that keeps growing along the keys."""
    d = Drafter([1200], 2, 128, FP16, seed=12)
    ramp = torch.linspace(0.1, 3, 1200, device="cuda", dtype=torch.float16)
    for e in range(5):
        k = min(PAGE, 1200 - e * PAGE)
        d.data[int(d.pool.tables[0, e]), :, 0, :k] = (ramp[e * PAGE:e * PAGE + k, None] *
                                                     torch.ones(128, device="cuda", dtype=torch.float16))
    q = d.rows(n, 4).abs()
    entries = [(0, 1200 - n, 0, n)]
    for scale in (0.5, 0.01):
        check(d, q, entries, call(d, q, entries, scale=scale), scale=scale)
        check(d, -q, entries, call(d, -q, entries, scale=scale), scale=scale)


@pytest.mark.parametrize("n", [1, 25])
def test_the_same_every_time_on_any_stream_and_from_graphs(gpu, n):
    """Captured once, replayed on other lengths and tables; two graphs share one workspace."""
    lens = [(5000, n), (33, n), (900, n)]
    entries, rows = ragged(lens)
    d = Drafter([c + n for c, _ in lens], 2, 128, BF16, seed=13)
    q = d.rows(rows, 8)
    shape, spec = stv.make_row_shape(8, 2, 128, BF16), stv.make_attn(window=700, sinks=9)
    ws = torch.empty(stv.stv_paged_attn_workspace_bytes(shape, n), dtype=torch.uint8, device="cuda")
    ctx, start = dev([c for c, _ in lens]), dev([0] + [e[2] + e[3] for e in entries])
    o, o2 = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    run = lambda out: stv.stv_paged_attn(shape, spec, d.layer, d.pool, None, ctx, start, n, q, out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(o)
    torch.cuda.current_stream().wait_stream(side)
    first = o.clone()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for gr, out in zip(graphs, (o, o2)):
        with torch.cuda.graph(gr):
            run(out)
    for _ in range(2):
        o.fill_(7.0)
        o2.fill_(7.0)
        for gr in graphs:
            gr.replay()
        assert torch.equal(o, first) and torch.equal(o2, first)
    ctx[0] = 1234
    graphs[0].replay()
    check(d, q, [(0, 1234, 0, n)] + entries[1:], o, window=700, sinks=9)


def test_many_short_sequences(gpu):
    rng = np.random.default_rng(14)
    lens = [(int(c), int(k)) for c, k in zip(rng.integers(0, 40, 300), rng.integers(0, 3, 300))]
    entries, n = ragged(lens)
    d = Drafter([c + k for c, k in lens], 1, 64, BF16, seed=14)
    q = d.rows(n, 4)
    check(d, q, entries, call(d, q, entries))
    check(d, q, entries, call(d, q, entries, max_new=9))


def test_offsets_past_32_bits(gpu):
    """A pool of more than 4 GiB whose last pages hold the sequence."""
    pages = 4200
    d = Drafter([], 4, 256, BF16, fill=0.0, n_pages=pages, max_seqs=1)
    assert d.data.numel() * 2 > 1 << 32
    n = 600
    d.pool.tables = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    d.pool = stv.PagePool(torch.zeros(pages, dtype=torch.int32, device="cuda"), dev([[pages - 1, pages - 3, pages - 2, -1]]), dev([3]))
    k, v = d.rows(n, 4), d.rows(n, 4)
    pos = np.arange(n)
    slots = np.array([pages - 1, pages - 3, pages - 2])[pos // PAGE] * PAGE + pos % PAGE
    shape = stv.make_row_shape(24, 4, 256, BF16)
    stv.stv_kv_write(shape, d.layer, k, v, dev(slots))
    kv = d.keys(0, n)
    assert torch.equal(kv[:, :, 0], k.double()) and torch.equal(kv[:, :, 1], v.double())
    q = d.rows(30, 24)
    entries = [(0, n - 30, 0, 30)]
    check(d, q, entries, call(d, q, entries))
    check(d, q[:1], [(0, n - 1, 0, 1)], call(d, q[:1].clone(), [(0, n - 1, 0, 1)]))


@pytest.mark.parametrize("n,ctx", [(1, 40), (1, 9000), (30, 40), (30, 9000)])
@pytest.mark.parametrize("hd", [64, 256])
def test_nan_goes_where_it_is_seen(gpu, n, ctx, hd):
    """A head of q that is NaN, and a key that is: the rows that see them and no others, whether
    or not their units are cut."""
    d = Drafter([ctx + n], 2, hd, BF16, seed=15)
    q = d.rows(n, 8)
    entries = [(0, ctx, 0, n)]
    clean = call(d, q, entries)
    bad = q.clone()
    bad[n - 1, 5] = float("nan")
    got = call(d, bad, entries)
    assert got[n - 1, 5].isnan().all()
    got[n - 1, 5] = clean[n - 1, 5]
    assert torch.equal(got, clean)
    if n > 1:  # the last token's key: its own row sees it
        pos = ctx + n - 1
        d.data[int(d.pool.tables[0, pos // PAGE]), 1, 0, pos % PAGE] = float("nan")
        got = call(d, q, entries)
        assert got[n - 1, 4:].isnan().all()
        got[n - 1, 4:] = clean[n - 1, 4:]
        assert torch.equal(got, clean)


def test_entries_that_share_rows(gpu):
    """More tiles of rows than there are rows: nothing is written."""
    d = Drafter([300] * 60, 1, 64, BF16, seed=16)
    q = d.rows(8, 128)
    shape = stv.make_row_shape(128, 1, 64, BF16)
    ws = torch.empty(stv.stv_paged_attn_workspace_bytes(shape, 8), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    stv.stv_paged_attn(shape, stv.make_attn(), d.layer, d.pool, None, dev([200] * 60), dev([0, 8] * 30 + [0]), 8, q, o, ws,
                       status)
    assert status.item() == stv.STV_DEV_BAD_ROW and (o == 7.0).all()


@pytest.mark.parametrize("max_new", [2, 40])
def test_a_sequence_twice_in_the_list(gpu, max_new):
    d = Drafter([700, 90], 2, 128, BF16, seed=17)
    q = d.rows(6, 8)
    q[4:] = q[:2]
    entries = [(0, 698, 0, 2), (1, 88, 2, 2), (0, 698, 4, 2)]
    o = call(d, q, entries, max_new=max_new)
    check(d, q, entries, o)


@pytest.mark.parametrize("max_new", [1, 20])
def test_the_most_entries(gpu, max_new):
    """4,096 entries, most without rows, on the two kernels; one more is refused."""
    rng = np.random.default_rng(18)
    lens = [(int(c), int(k)) for c, k in zip(rng.integers(0, 30, 4096), rng.random(4096) < 0.2)]
    lens[4095] = (2500, 1)
    entries, n = ragged(lens)
    d = Drafter([c + k if k else 0 for c, k in lens], 1, 64, FP16, seed=18)
    q = d.rows(n, 2)
    check(d, q, entries, call(d, q, entries, max_new=max_new))


@pytest.mark.parametrize("n", [1, 20])
def test_windows_and_first_tokens_without_end(gpu, n):
    """The largest window sees what no window does; so do the most first tokens."""
    d = Drafter([900 + n], 2, 64, FP16, seed=19)
    q = d.rows(n, 8)
    entries = [(0, 900, 0, n)]
    want = call(d, q, entries)
    most = (1 << 31) - 1
    assert torch.equal(call(d, q, entries, window=most), want)
    assert torch.equal(call(d, q, entries, window=most, sinks=most), want)
    check(d, q, entries, call(d, q, entries, window=3, sinks=most), window=3, sinks=most)


@pytest.mark.parametrize("n", [1, 40])
def test_two_calls_at_once(gpu, n):
    """Two streams, a workspace each."""
    lens = [(6000, n), (50, n)]
    entries, rows = ragged(lens)
    d = Drafter([c + n for c, _ in lens], 2, 128, BF16, seed=20)
    qs = [d.rows(rows, 8) for _ in range(2)]
    want = [call(d, q, entries) for q in qs]
    shape, spec = stv.make_row_shape(8, 2, 128, BF16), stv.make_attn()
    ws = [torch.empty(stv.stv_paged_attn_workspace_bytes(shape, n), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ctx, start = dev([c for c, _ in lens]), dev([0, n, 2 * n])
    outs = [torch.full_like(q, 7.0) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                stv.stv_paged_attn(shape, spec, d.layer, d.pool, None, ctx, start, n, qs[i], outs[i], ws[i])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_a_long_flat_tail_counts(gpu, n, dtype):
    """One key far ahead of 100,000 equal ones, each 2^-26 of it: together 1.5e-3."""
    length = 100000
    d = Drafter([length], 1, 64, dtype, seed=21, fill=0.0)
    for e in range(-(-length // PAGE)):
        page = int(d.pool.tables[0, e])
        d.data[page, 0, 0] = 0
        d.data[page, 0, 1] = 1.0
    d.data[int(d.pool.tables[0, 0]), 0, 0, 7] = 1.0
    d.data[int(d.pool.tables[0, 0]), 0, 1, 7] = 0.0
    q = torch.ones((n, 2, 64), dtype=dtype, device="cuda")
    got = call(d, q, [(0, length - n, 0, n)], scale=26 * np.log(2.0) / 64).double()
    tail = (length - n + torch.arange(1, n + 1, device="cuda").double() - 1) * 2.0 ** -26
    want = (tail / (1 + tail))[:, None, None]
    # P (2^-26 and 1) is exact in both types, the result rounded; 26 ln 2 log2(e) / 64 in fp32, and fp32 sums
    # of up to 100,000 equal numbers
    tol = want * (torch.finfo(dtype).eps / 2 + 26 * 2.0 ** -22 + length * 2.0 ** -24)
    assert ((got - want).abs() <= tol).all()


# ------------------------------------------------------------ stv_kv_write --

@pytest.mark.parametrize("hkv,hd,dtype", [(4, 256, FP16), (1, 64, BF16), (3, 128, BF16)])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
def test_write(gpu, hkv, hd, dtype, layout):
    n = 333
    d = Drafter([], hkv, hd, dtype, fill=3.0, n_pages=5)
    if layout == "plain":
        k, v = d.rows(n, hkv), d.rows(n, hkv)
    elif layout == "fused":
        row = d.rows(n, 2 * hkv + 5)
        k, v = row[:, 5:5 + hkv], row[:, 5 + hkv:]
    else:
        flat = torch.randn((n, 2 * hkv * (hd + 1) + 1), device="cuda").to(dtype)
        k, v = (flat[:, 1 + i * hkv * (hd + 1):1 + (i + 1) * hkv * (hd + 1)].unflatten(1, (hkv, hd + 1))[:, :, :hd]
                for i in range(2))
    slots = np.random.default_rng(1).permutation(5 * PAGE)[:n]
    slots[[3, 77]] = -1
    slots[[5, 100]] = 5 * PAGE, -2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stv.stv_kv_write(stv.make_row_shape(hkv, hkv, hd, dtype), d.layer, k, v, dev(slots), dev_status=status)
    assert status.item() == stv.STV_DEV_BAD_PAGE
    want = torch.full_like(d.data, 3.0)
    for r, s in enumerate(slots.tolist()):
        if 0 <= s < 5 * PAGE:
            want[s // PAGE, :, 0, s % PAGE], want[s // PAGE, :, 1, s % PAGE] = k[r], v[r]
    assert torch.equal(d.data, want)


def test_write_nothing(gpu):
    d = Drafter([], 2, 64, BF16, fill=1.0, n_pages=2)
    e = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    stv.stv_kv_write(stv.make_row_shape(2, 2, 64, BF16), d.layer, e, e, dev([]))
    assert (d.data == 1.0).all()
