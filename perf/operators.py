"""Cases and plain forms of the operators around a verify round: rotary
positions with several axes, sampling from the target's logits, and the pages
of the paged cache (fork, reserve, free, compact).

``own = False``: plain torch forms.  ``own = True``: the library's calls.
"""
import numpy as np
import torch

own = False

PAGE_TOKENS = 256
# Bytes of one KV head's block in a page: the 3-bit and the K 4 / V 2-bit
# caches, and the int4 cache (include/stv.h).
HEAD_BLOCK = {"bit3": 57344, "int4": 66560, "k4v2": 57344}
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def _lib():
    import speculative_tree_verify_bit_gb300 as stv

    return stv


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _sample(name, n_seqs, nodes, vocab, dtype, params, pad=0, masked=0.0):
    return {"name": name, "op": "sample", "n_seqs": n_seqs, "nodes": nodes, "vocab": vocab, "dtype": dtype,
            "params": params, "pad": pad, "masked": masked}


def _rope(name, rows, dtype, rd, layout, fused, inverse, hq=24, hkv=4, head_dim=256):
    return {"name": name, "op": "rope", "rows": rows, "dtype": dtype, "rd": rd, "layout": layout, "fused": fused,
            "inverse": inverse, "hq": hq, "hkv": hkv, "head_dim": head_dim}


def _fork(name, n_src, copies, ctx_lo, layers, fmt="bit3"):
    return {"name": name, "op": "fork", "n_src": n_src, "copies": copies, "ctx_lo": ctx_lo, "layers": layers,
            "fmt": fmt, "hkv": 4}


def _compact(name, n_pages, n_seqs, live, layers, fmt="bit3"):
    return {"name": name, "op": "compact", "n_pages": n_pages, "n_seqs": n_seqs, "live": live, "layers": layers,
            "fmt": fmt, "hkv": 4}


def listed():
    return [
        # the next token of one chat answer: one row of the full vocabulary, nucleus sampling
        _sample("sample-one-row", 1, 1, 248320, "fp32", "top_p"),
        # one verify round: the 16 nodes of one request's token tree, the usual chat filters
        _sample("sample-tree-16", 1, 16, 248320, "bf16", "chat"),
        # eight requests' trees in one batch, each request with filters of its own
        _sample("sample-trees-8x16", 8, 16, 248320, "fp16", "mixed"),
        # a full batch (64 requests, 8-row trees), logits in 32 bits, filters of every kind
        _sample("sample-batch-64x8", 64, 8, 248320, "fp32", "mixed"),
        # constrained decoding: a small odd vocabulary in padded rows, most tokens masked to -inf
        _sample("sample-masked-37", 37, 1, 32003, "bf16", "mixed", pad=5, masked=0.7),
        # a verify round's 16 tree rows, partial rotary (64 of 256 channels), text positions ctx + depth
        _rope("rope-tree-16", 16, "fp16", 64, "sections", False, False),
        # an image/video prompt in q|k|v rows as the projection leaves them, axes interleaved over the pairs
        _rope("rope-video-5003", 5003, "bf16", 64, "interleaved", True, False),
        # a 32K-token text prompt, every channel rotated
        _rope("rope-prompt-32k", 32768, "fp16", 256, "sections", False, False),
        # the gradient of 4,097 rows in 32 bits (the inverse rotation)
        _rope("rope-grad-4097", 4097, "fp32", 128, "sections", False, True),
        # a second sample of one 32K-token request in 16 layers: share its pages, copy the last, reserve the round's
        _fork("fork-one", 1, 1, 32868, 16),
        # eight requests (1K and up), four samples each
        _fork("fork-8x4", 8, 4, 1024 + 77, 16),
        # a fragmented pool after a batch of requests has ended: live pages move to the front
        _compact("compact-768", 768, 12, 0.5, 16),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["sample", "rope", "fork", "compact"])
    if op == "sample":
        vocab = log_int(1000, 262144)
        nodes = rng.randint(1, 32)
        most = max(1, int(512 * 248320 * 4 / 4 / vocab) // nodes)
        n_seqs = log_int(1, max(2, min(64, most)))
        n_seqs = min(n_seqs, max(1, most))
        return {k: v for k, v in _sample("", n_seqs, nodes, vocab, rng.choice(list(DTYPES)),
                                         rng.choice(["top_p", "chat", "mixed", "plain"]), rng.choice([0, 0, 1, 13]),
                                         rng.choice([0.0, 0.0, 0.3, 0.9])).items() if k != "name"}
    if op == "rope":
        dtype = rng.choice(list(DTYPES))
        hd = rng.choice([64, 128, 256])
        rd = rng.choice([r for r in (32, 64, 96, 128, 256) if r <= hd])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.randint(1, 6)
        most = int(32768 * 28 * 256 * 2 / ((hq + hkv) * hd * ESIZE[dtype]))
        return {k: v for k, v in _rope("", log_int(1, min(40000, most)), dtype, rd,
                                       rng.choice(["sections", "interleaved"]), rng.random() < 0.5,
                                       rng.random() < 0.4, hq, hkv, hd).items() if k != "name"}
    if op == "fork":
        n_src = rng.randint(1, 8)
        return {k: v for k, v in _fork("", n_src, rng.randint(1, 4), rng.randint(1, 4096), rng.randint(1, 16),
                                       rng.choice(list(HEAD_BLOCK))).items() if k != "name"}
    layers = rng.randint(1, 16)
    return {k: v for k, v in _compact("", log_int(32, 640), rng.randint(2, 16), 0.2 + 0.6 * rng.random(), layers,
                                      rng.choice(list(HEAD_BLOCK))).items() if k != "name"}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1_000_003 + 5)
    return g


def _prepare_sample(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed + 11)
    n, v = case["n_seqs"] * case["nodes"], case["vocab"]
    # a broad bulk and a few tokens that the model favours
    buf = torch.empty((n, v + case["pad"]), device="cuda", dtype=DTYPES[case["dtype"]])
    at = 0
    while at < n:  # in blocks of rows, so that the 32-bit draw stays small
        m = min(64, n - at)
        x = 2.5 * torch.randn((m, v), generator=g, device="cuda")
        liked = torch.randint(0, v, (m, 48), generator=g, device="cuda")
        x.scatter_add_(1, liked, 12.0 * torch.rand((m, 48), generator=g, device="cuda"))
        if case["masked"]:
            drop = torch.rand((m, v), generator=g, device="cuda") < case["masked"]
            drop[:, v // 2] = False  # one token is always allowed
            x.masked_fill_(drop, -float("inf"))
        buf[at:at + m, :v] = x.to(buf.dtype)
        buf[at:at + m, v:] = 0
        at += m
    if case["masked"] and n > 1:  # a row with one token left
        buf[1, :v] = -float("inf")
        buf[1, v // 2] = 1.0
    s = case["n_seqs"]
    t = np.full(s, 0.7, np.float32)
    k = np.zeros(s, np.int32)
    p = np.full(s, 0.9, np.float32)
    m = np.zeros(s, np.float32)
    if case["params"] == "chat":
        t[:], k[:], p[:], m[:] = 0.8, 50, 0.95, 0.02
    elif case["params"] == "plain":
        t[:], p[:] = 1.0, 1.0
    elif case["params"] == "mixed":
        t = rng.choice(np.array([0.0, 0.5, 0.8, 1.0, 1.3], np.float32), s)
        k = rng.choice(np.array([0, 0, 20, 50, 1000], np.int32), s)
        p = rng.choice(np.array([0.8, 0.95, 1.0], np.float32), s)
        m = rng.choice(np.array([0.0, 0.0, 0.05], np.float32), s)
    dev = lambda a: torch.as_tensor(a, device="cuda")
    st = {"logits": buf[:, :v], "temperature": dev(t), "top_k": dev(k), "top_p": dev(p), "min_p": dev(m),
          "u": torch.rand(n, generator=g, device="cuda"), "nodes": case["nodes"],
          "ids": torch.empty(n, dtype=torch.int32, device="cuda"),
          "logprob": torch.empty(n, dtype=torch.float32, device="cuda")}
    return st


def _sections(rd, axes=3):
    """rd / 2 pairs over time, height and width."""
    h = rd // 2
    w = h * 10 // 32
    return [h - 2 * w, w, w]


def _pair_axes(rd, layout):
    """The axis of each pair: whole sections in turn, or the axes dealt one
    pair at a time (time takes the rest when height and width are used up)."""
    sec = _sections(rd)
    if layout == "sections":
        return [a for a, n in enumerate(sec) for _ in range(n)]
    out = []
    for i in range(rd // 2):
        a = i % 3
        out.append(a if a and i < 3 * sec[a] else 0)
    return out


def _prepare_rope(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed + 12)
    n, hq, hkv, hd, dt = case["rows"], case["hq"], case["hkv"], case["head_dim"], DTYPES[case["dtype"]]
    if case["fused"]:  # q | k | v in one row
        row = torch.randn((n, (hq + 2 * hkv) * hd), generator=g, device="cuda").to(dt)
        q, k = row[:, :hq * hd].unflatten(1, (hq, hd)), row[:, hq * hd:(hq + hkv) * hd].unflatten(1, (hkv, hd))
    else:
        q = torch.randn((n, hq, hd), generator=g, device="cuda").to(dt)
        k = torch.randn((n, hkv, hd), generator=g, device="cuda").to(dt)
    base = int(rng.integers(0, 262144 - 64))
    if case["layout"] == "sections":  # text: the same position on every axis (a tree's rows: ctx + depth)
        pos = base % 4096 + np.arange(n) if n > 32 else base + np.minimum(np.arange(n), rng.integers(1, 9))
        pos = np.stack([pos, pos, pos])
    else:  # frames of 24 x 40 patches
        i = np.arange(n)
        pos = np.stack([i // 960, i // 40 % 24, i % 40]) + base % 8192
    st = {"q": q, "k": k, "pos": torch.as_tensor(pos.astype(np.int32), device="cuda"),
          "q_out": torch.empty((n, hq, hd), device="cuda", dtype=dt),
          "k_out": torch.empty((n, hkv, hd), device="cuda", dtype=dt),
          "inverse": case["inverse"], "rd": case["rd"], "theta": 1.0e7,
          "axes": _pair_axes(case["rd"], case["layout"])}
    if own:
        st["spec"] = _lib().make_rope(case["rd"], _sections(case["rd"]), theta=st["theta"],
                                      interleaved=case["layout"] == "interleaved")
    return st


def _pool(case, n_pages, max_seqs, stride, seed):
    """An empty page pool over `layers` layers' caches, one buffer for all."""
    page_bytes = case["hkv"] * HEAD_BLOCK[case["fmt"]]
    data = torch.empty((case["layers"], n_pages, page_bytes // 4), dtype=torch.int32, device="cuda")
    data.random_(-2**31, 2**31 - 1, generator=_gen(seed))
    return {"data": data, "n_pages": n_pages, "T": 16,
            "refs": np.zeros(n_pages, np.int32), "tables": np.full((max_seqs, stride), -1, np.int32),
            "counts": np.zeros(max_seqs, np.int32), "ctx": np.zeros(max_seqs, np.int32)}


def _finish_pool(case, st):
    for name in ("refs", "tables", "counts", "ctx"):
        st[name] = torch.as_tensor(st[name], device="cuda")
    if own:
        stv = _lib()
        group = stv.GROUP_INT4 if case["fmt"] == "int4" else stv.GROUP
        kv = stv.STV_KV_K4V2 if case["fmt"] == "k4v2" else stv.STV_KV_BY_GROUP
        st["shape"] = stv.make_shape(24, case["hkv"], group, kv)
        flat = st["data"].view(torch.uint8)
        st["layers"] = [stv.LayerCache(flat[i].reshape(-1), case["hkv"], group) for i in range(case["layers"])]
        st["pool"] = stv.PagePool(st["refs"], st["tables"], st["counts"])
        st["ws"] = torch.empty(stv.stv_page_workspace_bytes(st["pool"]), dtype=torch.uint8, device="cuda")
    return st


def _fork_ctx(case, seed):
    """Contexts of the forked requests, and of the pages they need with a round's rows."""
    rng = np.random.default_rng(seed + 13)
    ctx = np.array([case["ctx_lo"] * (1 + i) + int(rng.integers(0, 200)) for i in range(case["n_src"])], np.int64)
    pages = -(-(ctx + 16) // PAGE_TOKENS)
    return ctx, pages


def _prepare_fork(case, seed):
    ctx, pages = _fork_ctx(case, seed)
    n_src, copies = case["n_src"], case["copies"]
    most = [-(-(case["ctx_lo"] * (1 + i) + 200 + 16) // PAGE_TOKENS) for i in range(n_src)]  # of any seed
    n_pages = sum(most) + n_src * copies * 2 + 8
    st = _pool(case, n_pages, n_src * (1 + copies), max(most) + 1, seed)
    perm = np.random.default_rng(seed + 14).permutation(n_pages)
    at = 0
    for s in range(n_src):
        mine = perm[at:at + pages[s]]
        at += pages[s]
        st["tables"][s, :pages[s]], st["counts"][s], st["ctx"][s] = mine, pages[s], ctx[s]
        st["refs"][mine] = 1
    st = _finish_pool(case, st)
    src = np.repeat(np.arange(n_src, dtype=np.int32), copies)
    st["src"] = torch.as_tensor(src, device="cuda")
    st["dst"] = torch.arange(n_src, n_src * (1 + copies), dtype=torch.int32, device="cuda")
    return st


def _prepare_compact(case, seed):
    n_pages, n_seqs = case["n_pages"], case["n_seqs"]
    st = _pool(case, n_pages, n_seqs, n_pages, seed)
    rng = np.random.default_rng(seed + 15)
    live = rng.permutation(n_pages)[:int(n_pages * case["live"])]
    cuts = np.sort(rng.integers(0, live.size + 1, n_seqs - 1))
    for s, part in enumerate(np.split(live, cuts)):
        if s and st["counts"][s - 1]:  # the prompt's first page is shared with the request before
            part = np.concatenate([st["tables"][s - 1, :1], part])
        st["tables"][s, :part.size], st["counts"][s] = part, part.size
        st["refs"][part] += 1
    st = _finish_pool(case, st)
    st["refs0"], st["tables0"] = st["refs"].clone(), st["tables"].clone()
    st["map"] = torch.empty(n_pages, dtype=torch.int32, device="cuda")
    st["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    return {"case": case, **{"sample": _prepare_sample, "rope": _prepare_rope, "fork": _prepare_fork,
                             "compact": _prepare_compact}[case["op"]](case, seed)}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _plain_sample(st):
    """Order the row (largest first, the lower index first among equals),
    keep the top-k, of those the shortest head that holds top_p of their mass,
    of those the tokens with at least min_p of the largest's mass; the token
    is the first whose running mass exceeds u times the kept mass."""
    x = st["logits"].float()
    n, v = x.shape
    of_row = torch.arange(n, device=x.device) // st["nodes"]
    t, k, p, m = (st[name][of_row, None].double() for name in ("temperature", "top_k", "top_p", "min_p"))
    order = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = t == 0
    # running masses in 64 bits: the token hangs on which side of a border u falls
    w = torch.exp((order.values.double() - order.values[:, :1].double()) / torch.where(greedy, 1.0, t))
    rank = torch.arange(v, device=x.device)
    w = torch.where((k > 0) & (rank >= k), 0.0, w)
    run = torch.cumsum(w, 1)
    before = run - w
    w = torch.where((p >= 1) | (before < p * run[:, -1:]) | (rank == 0), w, 0.0)
    w = torch.where((w >= m) & ~(greedy & (rank > 0)), w, 0.0)
    run = torch.cumsum(w, 1)
    total = run[:, -1:]
    at = (run <= st["u"][:, None].double() * total).sum(1, keepdim=True)
    last = (w > 0).sum(1, keepdim=True) - 1
    at = torch.minimum(at, last)
    ids = torch.gather(order.indices, 1, at)[:, 0].to(torch.int32)
    logprob = torch.log(torch.gather(w, 1, at) / total)[:, 0].float()
    return [ids, logprob]


def _plain_rope(st):
    rd, h = st["rd"], st["rd"] // 2
    dev = st["q"].device
    # angles in 64 bits: a position of 262,144 times a frequency of 1 leaves few digits in 32
    freq = st["theta"] ** (-2.0 * torch.arange(h, device=dev, dtype=torch.float64) / rd)
    axes = torch.as_tensor(st["axes"], device=dev)
    angle = st["pos"].double()[axes].T * freq
    if st["inverse"]:
        angle = -angle
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    outs = []
    for x, out in ((st["q"], st["q_out"]), (st["k"], st["k_out"])):
        a, b = x[..., :h].float(), x[..., h:rd].float()
        out[..., :h] = (a * c - b * s).to(x.dtype)
        out[..., h:rd] = (b * c + a * s).to(x.dtype)
        out[..., rd:] = x[..., rd:]
        outs.append(out)
    return outs


def _lowest_free(refs, n):
    return torch.nonzero(refs == 0)[:n, 0]


def _plain_free(st, seqs):
    for s in seqs:
        n = int(st["counts"][s])
        mine = st["tables"][s, :n].long()
        st["refs"][mine] -= 1
        st["tables"][s, :n] = -1
        st["counts"][s] = 0


def _plain_fork(st):
    src, dst = st["src"].tolist(), st["dst"].tolist()
    _plain_free(st, dst)
    for a, b in zip(src, dst):
        ctx = int(st["ctx"][a])
        full = ctx // PAGE_TOKENS
        pages = st["tables"][a, :full]
        st["tables"][b, :full] = pages
        st["refs"][pages.long()] += 1
        st["counts"][b] = full
        st["ctx"][b] = ctx
        if ctx % PAGE_TOKENS:  # the last page goes on being written: a copy
            new = _lowest_free(st["refs"], 1)
            st["data"][:, new] = st["data"][:, st["tables"][a, full:full + 1].long()]
            st["tables"][b, full:full + 1] = new.to(torch.int32)
            st["refs"][new] = 1
            st["counts"][b] = full + 1
    for b in dst:
        have = int(st["counts"][b])
        need = -(-(int(st["ctx"][b]) + st["T"]) // PAGE_TOKENS)
        if need > have:
            new = _lowest_free(st["refs"], need - have)
            st["tables"][b, have:need] = new.to(torch.int32)
            st["refs"][new] = 1
            st["counts"][b] = need
    return [st["refs"], st["tables"], st["counts"], st["ctx"], st["data"]]


def _plain_compact(st):
    refs, tables = st["refs"], st["tables"]
    live = refs > 0
    n_live = live.sum()
    page = torch.arange(refs.numel(), device=refs.device)
    src = page[live & (page >= n_live)]
    dst = page[~live & (page < n_live)]
    st["data"][:, dst] = st["data"][:, src]
    to = torch.where(live, page, -1)
    to[src] = dst
    st["map"].copy_(to)
    moved = to[tables.clamp(min=0).long()].to(torch.int32)
    held = torch.arange(tables.shape[1], device=refs.device) < st["counts"][:, None]
    tables.copy_(torch.where(held, moved, tables))
    refs[dst] = refs[src]
    refs[src] = 0
    st["n_live"].copy_(n_live)
    return [refs, tables, st["map"], st["n_live"], st["data"]]


def run(st):
    op = st["case"]["op"]
    if op == "compact":  # the fragmented books of this state (the pages above stay as they were)
        st["refs"].copy_(st["refs0"])
        st["tables"].copy_(st["tables0"])
    if not own:
        return {"sample": _plain_sample, "rope": _plain_rope, "fork": _plain_fork,
                "compact": _plain_compact}[op](st)
    stv = _lib()
    if op == "sample":
        stv.stv_sample(st["logits"], st["u"], st["ids"], st["logprob"], temperature=st["temperature"],
                       top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"], rows_per_param=st["nodes"])
        return [st["ids"], st["logprob"]]
    if op == "rope":
        stv.stv_rope(st["spec"], st["pos"], st["q"], st["q_out"], st["k"], st["k_out"], inverse=st["inverse"])
        return [st["q_out"], st["k_out"]]
    if op == "fork":
        # the samples of the last round are freed, new ones forked, and the round's pages reserved
        stv.stv_page_free(st["pool"], st["dst"])
        stv.stv_page_fork(st["shape"], st["layers"], st["pool"], st["src"], st["dst"], st["ctx"], st["ws"])
        stv.stv_page_reserve(st["pool"], st["dst"], st["ctx"], st["T"])
        return [st["refs"], st["tables"], st["counts"], st["ctx"], st["data"]]
    stv.stv_page_compact(st["shape"], st["layers"], st["pool"], st["map"], st["n_live"], st["ws"])
    return [st["refs"], st["tables"], st["map"], st["n_live"], st["data"]]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "sample":
        n = case["n_seqs"] * case["nodes"]
        # an exponential (its range reduction and polynomial) and an addition for each token
        return {"bytes": n * case["vocab"] * ESIZE[case["dtype"]] + 12 * n, "flops": 10 * n * case["vocab"]}
    if op == "rope":
        heads = case["hq"] + case["hkv"]
        return {"bytes": case["rows"] * (2 * heads * case["head_dim"] * ESIZE[case["dtype"]] + 12),
                "flops": case["rows"] * case["rd"] // 2 * (6 * heads + 40)}
    page = case["hkv"] * HEAD_BLOCK[case["fmt"]] * case["layers"]
    if op == "fork":
        ctx, pages = _fork_ctx(case, 0)
        books = int(pages.sum()) * case["copies"] * 3 * 4 * 2
        return {"bytes": 2 * case["n_src"] * case["copies"] * page + books, "flops": 0}
    live = int(case["n_pages"] * case["live"])
    moved = live * (case["n_pages"] - live) // case["n_pages"]  # the live pages expected above the first `live`
    return {"bytes": 2 * moved * page + 4 * (3 * case["n_pages"] + 2 * live), "flops": 0}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def _exact_sample(case, seed):
    st = _prepare_sample(case, seed)
    ids, lps = [], []
    t, k, p, m, u = (st[name].cpu().numpy().astype(np.float64) for name in ("temperature", "top_k", "top_p",
                                                                             "min_p", "u"))
    for r in range(st["u"].numel()):
        s = r // case["nodes"]
        x = st["logits"][r].double()
        if t[s] == 0:
            ids.append(int(torch.nonzero(x == x.max())[0, 0]))
            lps.append(0.0)
            continue
        # a sort of (-x, index), without regard to the other form's
        val, idx = torch.sort(-x, stable=True)
        seen = int(torch.isfinite(val).sum())
        if k[s] > 0:
            seen = min(seen, int(k[s]))
        w = torch.exp((val[0] - val[:seen]) / t[s])
        run = w.cumsum(0)
        if p[s] < 1:
            keep = 1 + int((run < p[s] * run[-1]).sum())
            w = w[:min(keep, seen)]
        w = w[:max(1, int((w >= m[s]).sum()))]
        run = w.cumsum(0)
        at = min(int(torch.searchsorted(run, (u[r] * run[-1]).reshape(1), right=True)[0]), w.numel() - 1)
        ids.append(int(idx[at]))
        lps.append(float(torch.log(w[at] / run[-1])))
    return [np.array(ids, np.int32), np.array(lps, np.float64)]


def _exact_rope(case, seed):
    st = _prepare_rope(case, seed)
    h = case["rd"] // 2
    axes = np.array(_pair_axes(case["rd"], case["layout"]))
    pos = st["pos"].cpu().numpy().astype(np.float64)
    phi = pos[axes, :].T * np.power(1.0e7, -np.arange(h) / h)
    turn = torch.as_tensor(np.exp(1j * phi * (-1 if case["inverse"] else 1)), device="cuda")[:, None]
    out = []
    for x in (st["q"], st["k"]):
        y = x.double()
        z = torch.complex(y[..., :h], y[..., h:2 * h]) * turn
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
        out.append(y.cpu().numpy())
    return out


def exact(case, seed):
    if case["op"] == "sample":
        return _exact_sample(case, seed)
    if case["op"] == "rope":
        if case["rows"] * (case["hq"] + case["hkv"]) * case["head_dim"] > 1 << 28:
            return None
        return _exact_rope(case, seed)
    return None  # bytes and whole numbers
