"""The page calls against plain books (opkit.Books): refs, tables, counts and
ctx equal, and every page of every layer holding what the books say."""
import numpy as np
import pytest
import torch

import opkit
import speculative_tree_verify_bit_gb300 as stv

pytestmark = pytest.mark.gpu


class Kit:
    """A pool, its layers, and the same books on the host.  Page i of layer l
    starts out filled with words derived from (i, l)."""

    def __init__(self, n_pages=64, max_seqs=12, stride=16, layers=2, fmt="bit3", hkv=1, extra=3):
        group, kv = {"bit3": (32, 0), "int4": (256, 0), "k4v2": (32, stv.STV_KV_K4V2)}[fmt]
        self.shape = stv.make_shape(hkv * 6, hkv, group, kv)
        self.host = opkit.Books(n_pages, max_seqs, stride)
        self.pool = stv.PagePool.empty(n_pages, max_seqs, stride)
        self.ctx = torch.zeros(max_seqs, dtype=torch.int32, device="cuda")
        # a pool may be longer than the books: those pages are never touched
        self.layers = [stv.LayerCache.empty(n_pages + extra, hkv, group=group) for _ in range(layers)]
        for l in range(layers):
            w = self.words(l)
            w.copy_(torch.arange(1, w.shape[0] + 1, device="cuda")[:, None] * 64 + l +
                    131072 * torch.arange(w.shape[1], device="cuda"))
        self.ws = torch.full((stv.stv_page_workspace_bytes(self.pool),), 0xee, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def words(self, l):
        return self.layers[l].pool.view(torch.int32).view(self.layers[l].n_pages, -1)

    def set_ctx(self, ctx):
        self.host.ctx[:len(ctx)] = ctx
        self.ctx.copy_(torch.as_tensor(self.host.ctx, device="cuda"))

    def ids(self, v):
        return torch.as_tensor(np.asarray(v, np.int32), device="cuda")

    def reserve(self, seqs, extra):
        stv.stv_page_reserve(self.pool, self.ids(seqs), self.ctx, extra, dev_status=self.status)

    def fork(self, src, dst):
        stv.stv_page_fork(self.shape, self.layers, self.pool, self.ids(src), self.ids(dst), self.ctx, self.ws,
                          dev_status=self.status)

    def free(self, seqs):
        stv.stv_page_free(self.pool, self.ids(seqs), dev_status=self.status)

    def compact(self):
        m = torch.empty(self.pool.refs.numel(), dtype=torch.int32, device="cuda")
        n = torch.empty(1, dtype=torch.int32, device="cuda")
        stv.stv_page_compact(self.shape, self.layers, self.pool, m, n, self.ws, dev_status=self.status)
        return m.cpu().numpy(), int(n.item())

    def books(self):
        return [t.clone() for t in (self.pool.refs, self.pool.tables, self.pool.counts, self.ctx)]

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        h = self.host
        for got, want in zip(self.books(), (h.refs, h.tables, h.counts, h.ctx)):
            assert np.array_equal(got.cpu().numpy(), want)
        for l in range(len(self.layers)):
            w = self.words(l)
            first = np.concatenate([h.data, np.arange(h.data.size + 1, w.shape[0] + 1)])
            want = (torch.as_tensor(first, device="cuda")[:, None] * 64 + l +
                    131072 * torch.arange(w.shape[1], device="cuda")).to(torch.int32)
            assert torch.equal(w, want)


@pytest.mark.parametrize("fmt,hkv", [("bit3", 1), ("bit3", 4), ("int4", 1), ("int4", 4), ("k4v2", 2)])
def test_life_of_a_batch(gpu, fmt, hkv):
    """Reserve, fork, reserve, free, compact, and again in the compacted pool."""
    k = Kit(fmt=fmt, hkv=hkv)
    k.set_ctx([700, 256, 0, 1])
    k.reserve([0, 1, 2, 3], 16)
    k.host.reserve([0, 1, 2, 3], 16)
    k.check()
    k.fork([0, 0, 1, 2, 3], [4, 5, 6, 7, 8])  # partial, shared source, whole pages only, empty, one token
    k.host.fork([0, 0, 1, 2, 3], [4, 5, 6, 7, 8])
    k.check()
    k.reserve([8, 6, 5, 4, 7], 500)
    k.host.reserve([8, 6, 5, 4, 7], 500)
    k.check()
    k.fork([5], [9])
    k.host.fork([5], [9])
    k.free([0, 6, 3, 10])  # 10 holds nothing
    k.host.free([0, 6, 3, 10])
    k.check()
    where, n = k.compact()
    w2, n2 = k.host.compact()
    assert np.array_equal(where, w2) and n == n2
    k.check()
    where, n = k.compact()  # nothing left to move
    w2, n2 = k.host.compact()
    assert np.array_equal(where, w2) and n == n2
    k.reserve([0, 9], 900)
    k.host.reserve([0, 9], 900)
    k.free([1, 2, 4, 5, 7, 8, 9, 0])
    k.host.free([1, 2, 4, 5, 7, 8, 9, 0])
    k.check()
    assert int(k.pool.refs.count_nonzero().item()) == 0
    where, n = k.compact()
    assert n == 0 and (where == -1).all()


@pytest.mark.parametrize("seed", range(6))
def test_random_lives(gpu, seed):
    rng = np.random.default_rng(seed)
    n_pages = int(rng.integers(1, 200))
    k = Kit(n_pages=n_pages, max_seqs=int(rng.integers(2, 40)), stride=int(rng.integers(1, 30)),
            layers=int(rng.integers(1, 4)), extra=int(rng.integers(0, 2)))
    h = k.host
    m = h.counts.size
    for _ in range(25):
        op = rng.choice(["ctx", "reserve", "fork", "free", "compact"])
        seqs = rng.permutation(m)[:rng.integers(1, m + 1)].tolist()
        if op == "ctx":
            k.set_ctx([min(int(c * 256 * rng.random()), 32 * 256) if rng.random() < 0.7 else int(c) * 256
                       for c in h.counts])
        elif op == "reserve":
            extra = int(rng.integers(0, 700))
            need = sum(max(0, -(-(int(h.ctx[s]) + extra) // 256) - int(h.counts[s])) for s in seqs)
            ok = need <= len(h.free_pages()) and all((h.ctx[s] + extra + 255) // 256 <= h.tables.shape[1] for s in seqs)
            k.reserve(seqs, extra)
            if ok:
                h.reserve(seqs, extra)
            else:
                assert int(k.status.item()) != 0
                k.status.zero_()
        elif op == "fork":
            dst = [s for s in seqs if h.counts[s] == 0]
            src = [s for s in range(m) if s not in dst]
            if not src or not dst:
                continue
            src = rng.choice(src, len(dst)).tolist()
            ok = sum(int(h.ctx[s]) % 256 != 0 for s in src) <= len(h.free_pages()) and all(
                -(-int(h.ctx[s]) // 256) <= h.counts[s] for s in src)
            k.fork(src, dst)
            if ok:
                h.fork(src, dst)
            else:
                assert int(k.status.item()) != 0
                k.status.zero_()
        elif op == "free":
            k.free(seqs)
            h.free(seqs)
        else:
            where, n = k.compact()
            w2, n2 = h.compact()
            assert np.array_equal(where, w2) and n == n2
        k.check()


def test_wrong_calls_change_nothing(gpu):
    k = Kit(n_pages=10, max_seqs=6, stride=8)
    k.set_ctx([300, 600])
    k.reserve([0, 1], 0)
    k.host.reserve([0, 1], 0)
    S, P, N = stv.STV_DEV_BAD_SEQ, stv.STV_DEV_BAD_PAGE, stv.STV_DEV_NO_PAGES
    calls = [
        (lambda: k.reserve([0, 0], 400), S), (lambda: k.reserve([-1], 4), S), (lambda: k.reserve([6], 4), S),
        (lambda: k.reserve([0], 8 * 256), S),                     # more pages than a table row holds
        (lambda: k.reserve([0, 1, 2], 4 * 256 - 300), N),
        (lambda: k.reserve([0], 2 ** 31 - 1), S),
        (lambda: k.fork([0], [1]), S),                            # the destination holds pages
        (lambda: k.fork([0, 1], [2, 2]), S), (lambda: k.fork([2, 0], [3, 2]), S), (lambda: k.fork([3], [3]), S),
        (lambda: k.fork([6], [2]), S), (lambda: k.fork([0], [-1]), S),
        (lambda: k.free([0, 0]), S), (lambda: k.free([7]), S), (lambda: k.free([0, -1]), S),
    ]
    for call, bit in calls:
        k.status.zero_()
        call()
        k.check(status=bit)
    # a context past the pages held, a negative one
    for c in (3 * 256, -5):
        k.status.zero_()
        k.set_ctx([c, 600])
        k.fork([0], [2])
        k.check(status=S)
    k.status.zero_()
    k.reserve([0], 4)  # ctx -5
    k.check(status=S)
    k.set_ctx([300, 600])
    # five forks of a partial page with five pages left is one too many for six
    k.status.zero_()
    k.fork([0, 0, 1, 1], [2, 3, 4, 5])
    k.host.fork([0, 0, 1, 1], [2, 3, 4, 5])
    k.check()
    k.free([5])
    k.host.free([5])
    k.reserve([2], 256 * 2)
    k.host.reserve([2], 256 * 2)
    k.check()
    k.fork([0], [5])
    k.check(status=N)


def test_bad_table_entries(gpu):
    """Entries outside the pool, or of free pages, are caught before use."""
    P, S = stv.STV_DEV_BAD_PAGE, stv.STV_DEV_BAD_SEQ
    for bad in (-1, 10, 2 ** 31 - 1, -2 ** 31, 9):  # 9: a free page
        k = Kit(n_pages=10, max_seqs=6, stride=8)
        k.set_ctx([600])
        k.reserve([0], 0)
        k.host.reserve([0], 0)
        k.pool.tables[0, 1] = bad
        k.host.tables[0, 1] = bad
        k.fork([0], [1])
        k.check(status=P)
        k.status.zero_()
        k.free([0])
        k.check(status=P)
        k.status.zero_()
        # compact leaves the entry, moves the rest
        k.pool.refs[0], k.pool.refs[5] = 0, 1
        k.pool.tables[0, 0] = 5
        where, n = k.compact()
        assert n == 3 and int(k.status.item()) == P
        assert k.pool.tables[0, :3].tolist() == [0, bad, 2] and where[5] == 0
    k = Kit(n_pages=10, max_seqs=6, stride=8)
    k.pool.counts[3] = 9  # past the table
    k.free([3])
    torch.cuda.synchronize()
    assert int(k.status.item()) == S and int(k.pool.counts[3].item()) == 9


def test_pages_with_holders_outside_the_tables(gpu):
    """A page that the caller holds (a prefix cache) is live: it is not handed
    out, it moves in a compaction, and the map says where to."""
    k = Kit(n_pages=12, max_seqs=3, stride=8)
    k.pool.refs[7] = 1
    k.host.refs[7] = 1
    k.pool.refs[0] = 2
    k.host.refs[0] = 2
    k.set_ctx([512])
    k.reserve([0], 0)
    k.host.reserve([0], 0)
    k.check()
    assert k.host.tables[0, :2].tolist() == [1, 2]
    where, n = k.compact()
    k.host.compact()
    k.check()
    assert n == 4 and where[7] == 3 and where[0] == 0


@pytest.mark.parametrize("n_pages", [31, 32, 33, 1023, 1025, 33000, 262144])
def test_large_books(gpu, n_pages):
    """Books alone at every size of the free-page search (one page of bytes
    per layer would not fit: reserve and free touch no layer)."""
    rng = np.random.default_rng(n_pages)
    refs = (rng.random(n_pages) < 0.7).astype(np.int32)
    pool = stv.PagePool(torch.as_tensor(refs, device="cuda"),
                        torch.full((2, n_pages), -1, dtype=torch.int32, device="cuda"),
                        torch.zeros(2, dtype=torch.int32, device="cuda"))
    free = np.flatnonzero(refs == 0)
    a = free.size // 3
    ctx = torch.tensor([a * 256, (free.size - a) * 256], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    both = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    stv.stv_page_reserve(pool, both, ctx, 1, dev_status=status)
    assert int(status.item()) == stv.STV_DEV_NO_PAGES
    assert np.array_equal(pool.refs.cpu().numpy(), refs)
    status.zero_()
    stv.stv_page_reserve(pool, both, ctx, 0, dev_status=status)
    assert int(status.item()) == 0
    t = pool.tables.cpu().numpy()
    assert np.array_equal(t[1, :free.size - a], free[:free.size - a])
    assert np.array_equal(t[0, :a], free[free.size - a:]) and (t[0, a:] == -1).all()
    assert (pool.refs == 1).all()
    stv.stv_page_free(pool, both, dev_status=status)
    assert int(status.item()) == 0
    assert np.array_equal(pool.refs.cpu().numpy(), refs) and (pool.tables == -1).all()


def test_many_sequences(gpu):
    m = 4096
    pool = stv.PagePool.empty(9000, m, 4)
    ctx = torch.arange(m, dtype=torch.int32, device="cuda") % 500
    seqs = torch.randperm(m, device="cuda", dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stv.stv_page_reserve(pool, seqs, ctx, 12, dev_status=status)
    assert int(status.item()) == 0
    need = (ctx + 12 + 255) // 256
    assert torch.equal(pool.counts, need.to(torch.int32))
    order = pool.tables[seqs.long()]
    held = order[order >= 0]
    assert torch.equal(held, torch.arange(int(need.sum()), dtype=torch.int32, device="cuda"))
    stv.stv_page_free(pool, seqs, dev_status=status)
    assert int(status.item()) == 0 and not pool.refs.any() and not pool.counts.any()


def test_page_copy(gpu):
    k = Kit(n_pages=20, layers=3, extra=0)
    src, dst = [3, 3, 0, 19, 7], [1, 2, 18, 5, 11]
    stv.stv_page_copy(k.shape, k.layers, k.ids(src), k.ids(dst), k.ws, dev_status=k.status)
    for a, b in zip(src, dst):
        k.host.data[b] = k.host.data[a]
    k.check()
    for a, b in (([0, 1], [2, 2]), ([0, 1], [1, 2]), ([20], [1]), ([0], [-1]), ([4], [4])):
        k.status.zero_()
        stv.stv_page_copy(k.shape, k.layers, k.ids(a), k.ids(b), k.ws, dev_status=k.status)
        k.check(status=stv.STV_DEV_BAD_PAGE)
    k.status.zero_()
    stv.stv_page_copy(k.shape, k.layers, k.ids([]), k.ids([]), k.ws, dev_status=k.status)
    k.check()


def test_pages_in_a_graph(gpu):
    """Free, fork and reserve captured once and replayed: the books move on
    the device alone, and each replay ends where the last one did."""
    k = Kit(n_pages=40, max_seqs=6, stride=16, layers=2)
    k.set_ctx([700, 1000])
    k.reserve([0, 1], 16)
    k.host.reserve([0, 1], 16)
    src, dst = k.ids([0, 1, 1]), k.ids([2, 3, 5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        stv.stv_page_free(k.pool, dst, dev_status=k.status)
        stv.stv_page_fork(k.shape, k.layers, k.pool, src, dst, k.ctx, k.ws, dev_status=k.status)
        stv.stv_page_reserve(k.pool, dst, k.ctx, 30, dev_status=k.status)
    k.check()  # capturing ran nothing
    for _ in range(3):
        graph.replay()
    h = k.host
    h.fork([0, 1, 1], [2, 3, 5])
    h.reserve([2, 3, 5], 30)
    k.check()


def test_pages_python_refusals(gpu, monkeypatch):
    k = Kit()
    with pytest.raises(ValueError):
        stv.PagePool(k.pool.refs, k.pool.tables, k.pool.counts[:3])
    with pytest.raises(TypeError):
        stv.PagePool(k.pool.refs.long(), k.pool.tables, k.pool.counts)
    with pytest.raises(ValueError):
        stv.stv_page_reserve(k.pool, k.ids([0]), k.ctx[:2], 4)
    with pytest.raises(ValueError):
        stv.stv_page_fork(k.shape, k.layers, k.pool, k.ids([0, 1]), k.ids([2]), k.ctx, k.ws)
    with pytest.raises(stv.StvError) as e:
        stv.stv_page_fork(k.shape, k.layers, k.pool, k.ids([0]), k.ids([2]), k.ctx, k.ws[:64])
    assert e.value.status == stv.STV_ERR_WORKSPACE_TOO_SMALL
    assert stv.stv_page_workspace_bytes(64) == stv.stv_page_workspace_bytes(k.pool)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)  # a pool on another device than the current one
    with pytest.raises(ValueError):
        stv.stv_page_free(k.pool, k.ids([0]))


@pytest.mark.parametrize("m,stride", [(4096, 1 << 19), (2048, (1 << 20) + 1024)])
def test_totals_past_32_bits(gpu, m, stride):
    """Every sequence with 2^31 / m pages or more: their sum passes an int.
    The pool has far fewer pages, and no call changes anything."""
    n_pages = 100
    pool = stv.PagePool(torch.zeros(n_pages, dtype=torch.int32, device="cuda"),
                        torch.full((m, stride), -1, dtype=torch.int32, device="cuda"),
                        torch.zeros(m, dtype=torch.int32, device="cuda"))
    layers = [stv.LayerCache.empty(n_pages, 1)]
    ws = torch.empty(stv.stv_page_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seqs = torch.arange(m, dtype=torch.int32, device="cuda")
    ctx = torch.full((m,), stride * 256 - 16, dtype=torch.int32, device="cuda")

    def unchanged(bit, counts, contexts):
        assert int(status.item()) == bit
        status.zero_()
        assert not pool.refs.any() and torch.equal(pool.counts, counts) and torch.equal(ctx, contexts)
        for t in pool.tables.split(512):
            assert int(t.min().item()) == int(t.max().item()) == -1

    want = ctx.clone()
    stv.stv_page_reserve(pool, seqs, ctx, 16, dev_status=status)
    unchanged(stv.STV_DEV_NO_PAGES, torch.zeros_like(seqs), want)
    pool.counts.fill_(stride)  # tables that name pages over and over
    held = pool.counts.clone()
    stv.stv_page_free(pool, seqs, dev_status=status)
    unchanged(stv.STV_DEV_BAD_SEQ, held, want)
    pool.counts[1:] = 0  # one source, forked into all others
    held = pool.counts.clone()
    stv.stv_page_fork(stv.make_shape(6, 1), layers, pool, torch.zeros_like(seqs[1:]), seqs[1:], ctx, ws,
                      dev_status=status)
    unchanged(stv.STV_DEV_BAD_SEQ, held, want)


def big_books(n_pages):
    pool = stv.PagePool.empty(n_pages, 2, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.tensor([700, 0], dtype=torch.int32, device="cuda")
    return pool, status, one, ctx


def test_books_of_two_sizes_from_two_threads(gpu):
    """A call on large books is launched whatever size another thread's have."""
    from concurrent.futures import ThreadPoolExecutor

    def work(n_pages):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            pool, status, one, ctx = big_books(n_pages)
            for _ in range(3000):
                stv.stv_page_reserve(pool, one, ctx, 16, dev_status=status)
            stream.synchronize()
            assert int(status.item()) == 0 and pool.tables[0, :3].tolist() == [0, 1, 2]
            assert int(pool.counts[0].item()) == 3
        return True

    with ThreadPoolExecutor(2) as ex:
        assert all(ex.map(work, (262144, 170000)))


def test_books_of_two_sizes_in_a_graph(gpu):
    """A graph with calls on large and then smaller books replays both."""
    kits = [big_books(n) for n in (262144, 170000)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for pool, status, one, ctx in kits:
            stv.stv_page_reserve(pool, one, ctx, 16, dev_status=status)
    graph.replay()
    torch.cuda.synchronize()
    for pool, status, one, ctx in kits:
        assert int(status.item()) == 0 and pool.tables[0, :3].tolist() == [0, 1, 2]
