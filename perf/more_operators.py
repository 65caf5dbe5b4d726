"""Cases and plain forms of the drafter's side of a verify round: pages and
slots for a ragged batch of new tokens, K and V rows written to a 16-bit paged
cache, attention over it (single tokens, blocks and prompts; sliding window
with first tokens that stay visible), and the acceptance of drafted tokens by
the target's probabilities.

``own = False``: plain torch forms.  ``own = True``: the library's calls.
"""
import numpy as np
import torch

own = False

PAGE = 256
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def _lib():
    import speculative_tree_verify_bit_gb300 as stv

    return stv


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _extend(name, old, fresh, max_ctx, max_prompt):
    return {"name": name, "op": "extend", "old": old, "fresh": fresh, "max_ctx": max_ctx, "max_prompt": max_prompt}


def _write(name, rows, dtype, hkv=4, hd=256, fused=False, hq=24):
    return {"name": name, "op": "write", "rows": rows, "dtype": dtype, "hkv": hkv, "hd": hd, "fused": fused, "hq": hq}


def _attn(name, seqs, new, ctx_lo, ctx_hi, dtype, hq=24, hkv=4, hd=256, window=0, sinks=0, causal=True):
    return {"name": name, "op": "attn", "seqs": seqs, "new": new, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "dtype": dtype,
            "hq": hq, "hkv": hkv, "hd": hd, "window": window, "sinks": sinks, "causal": causal}


def _accept(name, seqs, nodes, vocab, dtype, tree, drafts, sharp):
    return {"name": name, "op": "accept", "seqs": seqs, "nodes": nodes, "vocab": vocab, "dtype": dtype, "tree": tree,
            "drafts": drafts, "sharp": sharp}


def listed():
    return [
        # the next step of 64 running requests: one token each, a page now and then
        _extend("extend-tokens-64", 64, 0, 32768, 0),
        # 24 running requests and 13 new prompts in the places of ended ones
        _extend("extend-prompts-37", 24, 13, 32768, 5000),
        # a drafter's block of 8 rows for 8 requests, K and V inside the projection's rows
        _write("write-blocks-8x8", 64, "bf16", fused=True),
        # a 32K-token prompt
        _write("write-prompt-32k", 32768, "fp16"),
        # the next token of one request at the full native context
        _attn("attn-token-262k", 1, 1, 262100, 262143, "fp16"),
        # the next token of 64 requests of unequal lengths, half as wide heads
        _attn("attn-tokens-64", 64, 1, 100, 16384, "bf16", hd=128),
        # a block drafter: 16 rows that see one another, a sliding window and 4 first tokens
        _attn("attn-blocks-8x16", 8, 16, 1024, 131072, "bf16", hd=128, window=4096, sinks=4, causal=False),
        # a long prompt through a sliding-window layer
        _attn("attn-prompt-32k-window", 1, 32768, 0, 0, "fp16", window=2048, sinks=16),
        # a prompt through a layer that sees everything
        _attn("attn-prompt-8k", 1, 8192, 0, 0, "bf16", hd=128),
        # one request's chain of 7 drafts
        _accept("accept-chain-8", 1, 8, 248320, "fp32", "chain", "replaced", 1.0),
        # 8 requests' trees whose siblings are distinct tokens
        _accept("accept-trees-8x16", 8, 16, 248320, "bf16", "tree", "distinct", 0.8),
        # 64 requests whose drafts come from a lookup (no draft distribution)
        _accept("accept-lookup-64x8", 64, 8, 248320, "fp32", "chain", "certain", 0.6),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["extend", "write", "attn", "attn", "attn", "accept"])
    if op == "extend":
        case = _extend("", log_int(1, 64), rng.randint(0, 13), log_int(256, 32768), log_int(1, 5000))
    elif op == "write":
        hkv, hd = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        case = _write("", log_int(1, min(65536, 32768 * 1024 // (hkv * hd))), rng.choice(["fp16", "bf16"]), hkv, hd,
                      rng.random() < 0.5, hkv * rng.randint(1, 8))
    elif op == "attn":
        hkv, hd = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8])
        window = rng.choice([0, 0, log_int(16, 4096)])
        sinks = rng.choice([0, 4, rng.randint(1, 100)]) if window else 0
        kind = rng.choice(["tokens", "blocks", "prompts"])
        if kind == "prompts":
            seqs = rng.randint(1, 4)
            new = log_int(33, int((1.5e12 / (2 * seqs * hq * hd)) ** 0.5) - 500)
            lo, hi = 0, rng.choice([0, 1000])
        else:
            seqs = log_int(1, 64 if kind == "tokens" else 16)
            new = rng.choice([1, 1, 1, 2]) if kind == "tokens" else rng.randint(3, 32)
            lo, hi = 0, log_int(64, min(131072, 262144 * 1024 // (seqs * hkv * hd)))
        case = _attn("", seqs, new, lo, hi, rng.choice(["fp16", "bf16"]), hq, hkv, hd, window, sinks,
                     kind != "blocks" or rng.random() < 0.5)
    else:
        drafts = rng.choice(["replaced", "distinct", "certain"])
        vocab = log_int(1000, 262144)
        nodes = rng.randint(1, 32)
        seqs = log_int(1, max(2, min(64, 64 * 8 * 248320 // (2 * vocab * nodes))))
        case = _accept("", seqs, nodes, vocab, rng.choice(list(DTYPES)), rng.choice(["chain", "tree"]), drafts,
                       0.3 + 0.7 * rng.random())
    return {k: v for k, v in case.items() if k != "name"}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1_000_003 + 7)
    return g


def _dev(a, dtype=np.int32):
    return torch.as_tensor(np.asarray(a, dtype), device="cuda")


def _books(held, max_seqs, stride, n_pages, rng):
    """Tables of sequences that hold so many pages each, taken from all over the pool."""
    tables, refs = np.full((max_seqs, stride), -1, np.int32), np.zeros(n_pages, np.int32)
    perm, at = rng.permutation(n_pages), 0
    for s, n in enumerate(held):
        tables[s, :n] = perm[at:at + n]
        refs[perm[at:at + n]] = 1
        at += n
    return {"refs": _dev(refs), "tables": _dev(tables), "counts": _dev(held)}


def _pool(st):
    return _lib().PagePool(st["refs"], st["tables"], st["counts"])


def _prepare_extend(case, seed):
    rng = np.random.default_rng(seed + 21)
    n_old, n_new = case["old"], case["fresh"]
    n = n_old + n_new
    ctx = np.concatenate([rng.integers(1, case["max_ctx"] + 1, n_old), np.zeros(n_new, np.int64)])
    ended = rng.integers(1, case["max_ctx"] + 1, n_new)  # what the ended requests held
    held = np.concatenate([-(-ctx[:n_old] // PAGE), -(-ended // PAGE)])
    order = rng.permutation(n)  # old and new requests in any order
    ctx, held, old = ctx[order], held[order], order < n_old
    new = np.where(old, 1, rng.integers(1, case["max_prompt"] + 1, n) if n_new else 1)
    stride = -(-(max(case["max_ctx"], case["max_prompt"]) + 1) // PAGE) + 1
    max_rows = n_old + n_new * case["max_prompt"]
    st = _books(held, n, stride, n * stride, rng)
    st.update(seqs=_dev(np.arange(n)), ended=_dev(np.nonzero(~old)[0]), n_new=_dev(new), ctx=_dev(ctx),
              row_start=_dev(np.zeros(n + 1)), row_seq=_dev(np.zeros(max_rows)), row_pos=_dev(np.zeros(max_rows)),
              slots=_dev(np.zeros(max_rows)))
    if own:
        st["pool"] = _pool(st)
    return st


def _prepare_write(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed + 22)
    n, hkv, hd, hq, dt = case["rows"], case["hkv"], case["hd"], case["hq"], DTYPES[case["dtype"]]
    n_pages = n // PAGE + 9
    st = {"data": torch.zeros((n_pages, hkv, 2, PAGE, hd), dtype=dt, device="cuda")}
    if case["fused"]:  # q | k | v in one row
        row = torch.randn((n, (hq + 2 * hkv) * hd), generator=g, device="cuda").to(dt).view(n, hq + 2 * hkv, hd)
        st["k"], st["v"] = row[:, hq:hq + hkv], row[:, hq + hkv:]
    else:
        st["k"], st["v"] = (torch.randn((n, hkv, hd), generator=g, device="cuda").to(dt) for _ in range(2))
    # runs of 8 to 500 adjacent slots (the sequences' new rows), from anywhere in the pool
    slots, perm = [], rng.permutation(n_pages)
    first = int(rng.integers(0, PAGE))
    flat = (perm[:, None].astype(np.int64) * PAGE + np.arange(PAGE)).reshape(-1)
    slots = flat[first:first + n].copy()
    slots[rng.integers(0, n, n // 50)] = -1  # rows of padding
    st["slots"] = _dev(slots)
    if own:
        stv = _lib()
        st["shape"], st["layer"] = stv.make_row_shape(hkv, hkv, hd, dt), stv.RowCache(st["data"])
    return st


def _attn_lengths(case, seed):
    rng = np.random.default_rng(seed + 23)
    lo, hi, n = case["ctx_lo"], case["ctx_hi"], case["seqs"]
    ctx = rng.integers(lo, hi + 1, n) if n == 1 or hi < 64 else np.exp(
        rng.uniform(np.log(max(lo, 1)), np.log(hi), n)).astype(np.int64)
    new = np.full(n, case["new"], np.int64)
    if n > 1 and case["new"] > 1:  # ragged: some sequences have fewer new rows
        # (the same for every seed: the outputs keep their shape)
        new = np.random.default_rng(n).integers(max(1, case["new"] // 2), case["new"] + 1, n)
        new[n // 2] = case["new"]
    return ctx, new


def _prepare_attn(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed + 24)
    n, hq, hkv, hd, dt = case["seqs"], case["hq"], case["hkv"], case["hd"], DTYPES[case["dtype"]]
    ctx, new = _attn_lengths(case, seed)
    held = -(-(ctx + new) // PAGE)
    most = n * (-(-(case["ctx_hi"] + case["new"]) // PAGE)) if n == 1 else int(held.sum())
    stride, n_pages = int(held.max()) + 1, most + 3
    st = _books(held, n, stride, n_pages, rng)
    data = torch.empty((n_pages, hkv, 2, PAGE, hd), dtype=dt, device="cuda")
    for i in range(0, n_pages, 64):
        part = data[i:i + 64]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.float32))
    gain = 1.0 + 2.0 * torch.rand((hkv, 1, hd), generator=g, device="cuda")  # channels of unequal size, as keys have
    data[:, :, 0] *= gain.to(dt)
    rows = int(new.sum())
    st.update(data=data, ctx=_dev(ctx), row_start=_dev(np.concatenate([[0], np.cumsum(new)])), rows=rows,
              lens=list(zip(ctx.tolist(), new.tolist())),
              q=torch.randn((rows, hq, hd), generator=g, device="cuda").to(dt),
              o=torch.zeros((rows, hq, hd), dtype=dt, device="cuda"))
    if own:
        stv = _lib()
        st["shape"], st["layer"] = stv.make_row_shape(hq, hkv, hd, dt), stv.RowCache(data)
        st["spec"] = stv.make_attn(window=case["window"], sinks=case["sinks"], causal=case["causal"])
        st["pool"] = _pool(st)
        st["ws"] = torch.zeros(stv.stv_paged_attn_workspace_bytes(st["shape"], case["new"]), dtype=torch.uint8,
                               device="cuda")
    return st


def _tree(case, rng):
    t = case["nodes"]
    if case["tree"] == "chain":
        return np.arange(-1, t - 1)
    parent = np.full(t, -1, np.int64)
    for i in range(1, t):  # ranked best first: most nodes hang near the root
        parent[i] = int(rng.integers(0, max(1, (i + 2) // 3)))
    return parent


def _prepare_accept(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed + 25)
    n, t, v, dt = case["seqs"], case["nodes"], case["vocab"], DTYPES[case["dtype"]]
    parent = np.stack([_tree(case, rng) for _ in range(n)])
    p = torch.empty((n * t, v), dtype=dt, device="cuda")
    q = torch.empty((n * t, v), dtype=dt, device="cuda") if case["drafts"] != "certain" else None
    ids = torch.zeros((n, t), dtype=torch.int32, device="cuda")
    for s in range(n):
        x = 2.0 * torch.randn((t, v), generator=g, device="cuda")
        x.scatter_add_(1, torch.randint(0, v, (t, 40), generator=g, device="cuda"),
                       14.0 * torch.rand((t, 40), generator=g, device="cuda"))
        y = case["sharp"] * x + (1 - case["sharp"]) * torch.randn((t, v), generator=g, device="cuda")
        p[s * t:(s + 1) * t] = torch.softmax(x, 1).to(dt)
        qs = torch.softmax(y, 1)
        if q is not None:
            q[s * t:(s + 1) * t] = qs.to(dt)
            qs = q[s * t:(s + 1) * t].float()
        kids = [np.nonzero(parent[s] == a)[0] for a in range(t)]
        most = max(len(k) for k in kids)
        if most:
            drawn = torch.multinomial(qs.double(), most, replacement=case["drafts"] != "distinct",
                                      generator=g).to(torch.int32)
            for a, k in enumerate(kids):
                if len(k):
                    ids[s, _dev(k, np.int64)] = drawn[a, :len(k)]
    return {"parent": _dev(parent), "ids": ids, "p": p, "q": q, "u": torch.rand((n, t), generator=g, device="cuda"),
            "n_commit": _dev(np.zeros(n)), "path": _dev(np.zeros((n, t))), "out_ids": _dev(np.zeros((n, t)))}


def prepare(case, seed):
    return {"case": case, **{"extend": _prepare_extend, "write": _prepare_write, "attn": _prepare_attn,
                             "accept": _prepare_accept}[case["op"]](case, seed)}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _plain_extend(st):
    refs, tables, counts = st["refs"], st["tables"], st["counts"]
    for s in st["ended"].tolist():
        k = int(counts[s])
        refs[tables[s, :k].long()] -= 1
        tables[s, :k] = -1
        counts[s] = 0
    seqs, new = st["seqs"].long(), st["n_new"]
    need = (st["ctx"][seqs] + new + PAGE - 1) // PAGE
    want = torch.clamp(need - counts[seqs], min=0)
    free = torch.nonzero(refs == 0)[:, 0]
    at = 0
    for s, have, k in zip(seqs.tolist(), counts[seqs].tolist(), want.tolist()):
        if k:
            tables[s, have:have + k] = free[at:at + k].to(torch.int32)
            refs[free[at:at + k]] = 1
            at += k
    counts[seqs] += want.to(torch.int32)
    start = st["row_start"]
    start[0] = 0
    start[1:] = torch.cumsum(new, 0)
    r = torch.arange(st["slots"].numel(), device=refs.device)
    i = torch.searchsorted(start[1:].long(), r, right=True)
    live = i < seqs.numel()
    i = i.clamp(max=seqs.numel() - 1)
    pos = st["ctx"][seqs[i]] + r - start[i]
    page = tables[seqs[i], torch.where(live, pos // PAGE, 0)]
    for name, x in (("row_seq", i), ("row_pos", pos), ("slots", page * PAGE + pos % PAGE)):
        st[name].copy_(torch.where(live, x, -1))
    return [st[k] for k in ("refs", "tables", "counts", "row_start", "row_seq", "row_pos", "slots")]


def _plain_write(st):
    live = torch.nonzero(st["slots"] >= 0)[:, 0]
    slot = st["slots"][live].long()
    st["data"][slot // PAGE, :, 0, slot % PAGE] = st["k"][live]
    st["data"][slot // PAGE, :, 1, slot % PAGE] = st["v"][live]
    return [st["data"]]


def _plain_attn(st):
    c = st["case"]
    hkv, hd, g, w = c["hkv"], c["hd"], c["hq"] // c["hkv"], c["window"]
    row = 0
    for s, (ctx, new) in enumerate(st["lens"]):
        end = ctx + new
        pages = st["tables"][s, :-(-end // PAGE)].long()
        step = max(16, min(new, (1 << 27) // (c["hq"] * (min(end, w + 512) if w else end))))
        for r0 in range(0, new, step):
            r1 = min(new, r0 + step)
            # the keys that some of these rows see: the first ones, and a range
            lo = max(0, ctx + r0 - w + 1) if w else 0
            hi = ctx + r1 if c["causal"] else end
            keys = torch.arange(lo, hi, device=pages.device)
            if w and lo:
                keys = torch.cat([torch.arange(min(c["sinks"], lo), device=pages.device), keys])
            kv = st["data"][pages[keys // PAGE], :, :, keys % PAGE].float()  # [keys][hkv][2][hd]
            pos = torch.arange(ctx + r0, ctx + r1, device=pages.device)[:, None]
            seen = keys <= pos if c["causal"] else torch.ones_like(keys <= pos)
            if w:
                seen &= (keys > pos - w) | (keys < c["sinks"])
            qs = st["q"][row + r0:row + r1].float().view(r1 - r0, hkv, g, hd)
            for h in range(hkv):
                x = torch.matmul(qs[:, h].reshape(-1, hd), kv[:, h, 0].T).view(r1 - r0, g, -1) * hd ** -0.5
                x = x.masked_fill(~seen[:, None], -float("inf"))
                x = torch.exp(x - x.amax(2, keepdim=True))
                x = torch.matmul(x, kv[:, h, 1]) / x.sum(2, keepdim=True)
                st["o"][row + r0:row + r1, h * g:(h + 1) * g] = x.to(st["o"].dtype)
        row += new
    return [st["o"]]


def _plain_accept(st):
    """At a node, its children in turn: the child's token is taken if u times
    the draft's share is below the target's; otherwise the target keeps what
    it has above the draft, as a share of that."""
    n, t = st["ids"].shape
    parent, ids, u = st["parent"].tolist(), st["ids"].tolist(), st["u"].double().tolist()
    for name in ("path", "out_ids"):
        st[name].fill_(-1)
    for s in range(n):
        at, depth = 0, 0
        st["path"][s, 0] = 0
        while True:
            r = st["p"][s * t + at].double()
            d = st["q"][s * t + at].double() if st["q"] is not None else None
            taken = -1
            for c in [i for i in range(at + 1, t) if parent[s][i] == at]:
                x = ids[s][c]
                dx = float(d[x]) if d is not None else 1.0
                if u[s][c] * dx < float(r[x]):
                    taken = c
                    break
                if d is not None:
                    left = torch.clamp(r - d, min=0)
                else:
                    left = r.clone()
                    left[x] = 0
                z = float(left.sum())
                if z > 0:
                    r = left / z
                if st["case"]["drafts"] == "distinct":
                    d[x] = 0
                    d = d / max(1e-300, float(d.sum()))
            if taken < 0:
                break
            st["out_ids"][s, depth] = ids[s][taken]
            depth += 1
            at = taken
            st["path"][s, depth] = at
        run = torch.cumsum(r, 0)
        st["out_ids"][s, depth] = torch.nonzero(run > u[s][0] * run[-1])[0, 0]
        st["n_commit"][s] = depth + 1
    return [st["n_commit"], st["path"], st["out_ids"]]


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"extend": _plain_extend, "write": _plain_write, "attn": _plain_attn, "accept": _plain_accept}[op](st)
    stv = _lib()
    if op == "extend":
        if st["ended"].numel():
            stv.stv_page_free(st["pool"], st["ended"])
        stv.stv_page_extend(st["pool"], st["seqs"], st["n_new"], st["ctx"], st["row_start"], st["row_seq"],
                            st["row_pos"], st["slots"])
        return [st[k] for k in ("refs", "tables", "counts", "row_start", "row_seq", "row_pos", "slots")]
    if op == "write":
        stv.stv_kv_write(st["shape"], st["layer"], st["k"], st["v"], st["slots"])
        return [st["data"]]
    if op == "attn":
        stv.stv_paged_attn(st["shape"], st["spec"], st["layer"], st["pool"], None, st["ctx"], st["row_start"],
                           case["new"], st["q"], st["o"], st["ws"])
        return [st["o"]]
    stv.stv_tree_accept_probs(st["parent"], st["ids"], st["p"], st["q"], st["u"], st["n_commit"], st["path"],
                              st["out_ids"], distinct=case["drafts"] == "distinct")
    return [st["n_commit"], st["path"], st["out_ids"]]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "extend":
        n = case["old"] + case["fresh"]
        stride = -(-(max(case["max_ctx"], case["max_prompt"]) + 1) // PAGE) + 1
        rows = case["old"] + case["fresh"] * case["max_prompt"]
        return {"bytes": 4 * n * stride + 24 * n + 12 * rows, "flops": 0}
    if op == "write":
        return {"bytes": case["rows"] * (4 * case["hkv"] * case["hd"] * ESIZE[case["dtype"]] + 4), "flops": 0}
    if op == "attn":
        ctx, new = _attn_lengths(case, 0)
        w, pairs, keys = case["window"], 0, 0
        for c, n in zip(ctx.tolist(), new.tolist()):
            pos = np.arange(c, c + n, dtype=np.int64)
            hi = pos + 1 if case["causal"] else np.full(n, c + n, np.int64)
            lo = np.maximum(0, pos - w + 1) if w else np.zeros(n, np.int64)
            first = np.minimum(case["sinks"], lo)
            pairs += int((hi - lo + first).sum())
            keys += int(hi[-1] - lo[0] + first[0])
        es = ESIZE[case["dtype"]]
        return {"bytes": es * case["hd"] * (2 * case["hkv"] * keys + 2 * case["hq"] * int(new.sum())),
                "flops": 4 * case["hd"] * case["hq"] * pairs}
    rows = 1 if case["drafts"] == "certain" else 2
    return {"bytes": case["seqs"] * (rows * case["vocab"] * ESIZE[case["dtype"]] + 24 * case["nodes"]),
            "flops": 2 * case["seqs"] * case["vocab"]}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def _exact_attn(case, seed):
    st = _prepare_attn(case, seed)
    hq, hkv, hd, w = case["hq"], case["hkv"], case["hd"], case["window"]
    out = torch.zeros((st["rows"], hq, hd), dtype=torch.float64, device="cuda")
    table = st["tables"].cpu().numpy()
    row = 0
    for s, (ctx, new) in enumerate(st["lens"]):
        end = ctx + new
        flat = st["data"][torch.as_tensor(table[s, :-(-end // PAGE)].astype(np.int64), device="cuda")]
        for j0 in range(0, new, 256):
            j = np.arange(j0, min(new, j0 + 256)) + ctx
            mask = np.zeros((j.size, end), bool) if not case["causal"] else None
            k = np.arange(end)
            mask = (k[None] <= j[:, None]) if case["causal"] else np.ones((j.size, end), bool)
            if w:
                mask &= (k[None] > j[:, None] - w) | (k[None] < case["sinks"])
            used = np.nonzero(mask.any(0))[0]
            sel = torch.as_tensor(used, device="cuda")
            hide = torch.as_tensor(~mask[:, used], device="cuda")
            for h in range(hq):
                kk = flat[:, h // (hq // hkv), 0].reshape(-1, hd)[sel].double()
                vv = flat[:, h // (hq // hkv), 1].reshape(-1, hd)[sel].double()
                z = st["q"][row + j0:row + j0 + j.size, h].double() @ kk.T / np.sqrt(hd)
                z[hide] = -float("inf")
                out[row + j0:row + j0 + j.size, h] = torch.softmax(z, 1) @ vv
        row += new
    return [out.cpu().numpy()]


def _exact_accept(case, seed):
    st = _prepare_accept(case, seed)
    n, t = case["seqs"], case["nodes"]
    parent, ids = st["parent"].cpu().numpy(), st["ids"].cpu().numpy()
    u = st["u"].cpu().numpy().astype(np.float64)
    n_commit, path, out = np.zeros(n, np.int32), np.full((n, t), -1, np.int32), np.full((n, t), -1, np.int32)
    for s in range(n):
        nodes = [0]
        while True:
            row = s * t + nodes[-1]
            mass = st["p"][row].float().cpu().numpy().astype(np.float64)  # the target's, up to `scale`
            scale, gone = 1.0, 0.0
            draft = None if st["q"] is None else st["q"][row].float().cpu().numpy().astype(np.float64)
            whole = 1.0 if draft is None or case["drafts"] != "distinct" else None
            found = None
            for c in np.nonzero(parent[s] == nodes[-1])[0]:
                if c == 0:
                    continue
                x = ids[s, c]
                share = 1.0 if draft is None else draft[x]
                if u[s, c] * share * scale < mass[x]:
                    found = c
                    break
                rest = mass.copy()
                if draft is None:
                    rest[x] = 0.0
                else:
                    rest = np.maximum(mass - scale * draft, 0.0)
                if rest.sum() > 0:
                    mass, scale = rest, rest.sum()
                if whole is None:
                    draft[x] = 0.0
                    draft = draft / max(1e-300, draft.sum())
            if found is None:
                break
            nodes.append(int(found))
        acc = np.cumsum(mass)
        m = len(nodes)
        n_commit[s] = m
        path[s, :m] = nodes
        out[s, :m - 1] = ids[s, nodes[1:]]
        out[s, m - 1] = int(np.searchsorted(acc, u[s, 0] * acc[-1], side="right"))
    return [n_commit, path, out]


def exact(case, seed):
    if case["op"] == "accept":
        return _exact_accept(case, seed)
    if case["op"] == "attn":
        w = work(case)
        if w["flops"] > 3e12:
            return None
        return _exact_attn(case, seed)
    return None  # whole numbers and bits copied
