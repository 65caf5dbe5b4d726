"""Host-side refusals of stv_page_extend, stv_kv_write, stv_paged_attn and
stv_tree_accept_probs: every argument is checked before anything is enqueued,
so they need no GPU.  Device addresses are dummies and never dereferenced."""
import ctypes

import pytest
import torch

import speculative_tree_verify_bit_gb300 as stv
from speculative_tree_verify_bit_gb300 import build as stv_build

D = 0x7f0000000000  # a dummy device address, 16-byte aligned
OK, BAD, SHAPE, SMALL = (stv.STV_OK, stv.STV_ERR_INVALID_ARG, stv.STV_ERR_SHAPE_UNSUPPORTED,
                         stv.STV_ERR_WORKSPACE_TOO_SMALL)
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    stv_build.build()
    return stv.load()


def shape(hq=24, hkv=4, hd=128, dtype=BF16, **kw):
    s = stv.make_row_shape(hq, hkv, hd, dtype)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def rows(data=D, row=4096, head=128, heads=4):
    return stv.stv_rows(data, row, head, heads)


def layer(s, pool=D + (1 << 40), n_pages=8, page_bytes=None):
    return stv.stv_layer_cache(pool, page_bytes if page_bytes is not None else s.hkv * 1024 * s.head_dim, n_pages)


ref = lambda v: None if v is None else ctypes.byref(v)


# ----------------------------------------------------------- the shape ------

@pytest.mark.parametrize("s,rc", [
    (shape(), OK), (shape(hd=64), OK), (shape(hd=256, dtype=torch.float16), OK), (shape(hq=128, hkv=1), OK),
    (shape(hd=96), SHAPE), (shape(hd=512), SHAPE), (shape(hq=25), SHAPE), (shape(hq=0), SHAPE), (shape(hkv=0), SHAPE),
    (shape(hq=129, hkv=1), SHAPE), (shape(group=32), SHAPE), (shape(page_tokens=128), SHAPE), (shape(kv_format=3), SHAPE),
    (shape(kv_format=6), SHAPE), (shape(hq=2050, hkv=1025), SHAPE),
])
def test_row_shapes(lib, s, rc):
    out = ctypes.c_int64()
    assert lib.stv_page_bytes(ctypes.byref(s), ctypes.byref(out)) == rc
    if rc == OK:
        assert out.value == s.hkv * 2 * 256 * s.head_dim * 2


def test_the_quantized_calls_refuse_the_row_cache(lib):
    s = shape(hd=256)
    l = layer(s)
    seqs = (stv.stv_seq * 1)(stv.stv_seq(D, 4, 100))
    out = ctypes.c_size_t()
    assert lib.stv_verify_workspace_bytes(ref(s), seqs, 1, 1, 152, ctypes.byref(out)) == SHAPE
    assert lib.stv_kv_append_pack(ref(s), ref(l), seqs, 1, D, D, D, D, 1, None, None) == SHAPE
    assert lib.stv_verify_attn(ref(s), ref(l), seqs, 1, D, D, 1, 0, D, 1 << 30, None, None) == SHAPE
    q = stv.make_shape()
    assert lib.stv_kv_write(ref(q), ref(l), ref(rows()), ref(rows()), D, 1, None, None) == SHAPE


# ----------------------------------------------------- stv_page_extend ------

@pytest.mark.parametrize("kw,rc", [
    (dict(refs=None), BAD), (dict(n=-1), BAD), (dict(n=5), BAD), (dict(n_new=None), BAD), (dict(ctx=None), BAD),
    (dict(row_start=None), BAD), (dict(max_rows=-1), BAD), (dict(max_rows=(1 << 26) + 1), SHAPE),
    (dict(n_pages=0), BAD), (dict(n_pages=(1 << 18) + 1), SHAPE), (dict(max_seqs=4097), SHAPE),
])
def test_extend_refusals(lib, kw, rc):
    a = dict(refs=D, n_pages=8, max_seqs=4, seqs=D, n=4, n_new=D, ctx=D, row_start=D, maps=D, max_rows=16)
    a.update(kw)
    pool = stv.stv_page_pool(a["refs"], D, D, a["n_pages"], a["max_seqs"], 8)
    assert lib.stv_page_extend(ref(pool), a["seqs"], a["n"], a["n_new"], a["ctx"], a["row_start"], a["maps"], a["maps"],
                               a["maps"], a["max_rows"], None, None) == rc
    assert lib.stv_page_extend(None, a["seqs"], a["n"], a["n_new"], a["ctx"], a["row_start"], a["maps"], a["maps"],
                               a["maps"], a["max_rows"], None, None) == BAD


# -------------------------------------------------------- stv_kv_write ------

@pytest.mark.parametrize("kw,rc", [
    (dict(n=0), OK), (dict(n=-1), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(slots=None), BAD),
    (dict(k=rows(heads=3)), BAD), (dict(v=rows(heads=5)), BAD), (dict(k=rows(D + 1)), BAD), (dict(k=rows(0)), BAD),
    (dict(k=rows(head=64)), BAD), (dict(v=rows(row=256)), BAD), (dict(k=rows(row=1 << 46), n=1 << 20), BAD),
    (dict(l=layer(shape(), pool=0)), BAD), (dict(l=layer(shape(), pool=D + 8)), BAD), (dict(l=layer(shape(), n_pages=0)), BAD),
    (dict(l=layer(shape(), page_bytes=4096)), SHAPE), (dict(l=layer(shape(), n_pages=1 << 20)), SHAPE),
    (dict(k=rows(D + (1 << 40) + 4096)), BAD), (dict(v=rows(D + (1 << 40) + 8 * 4 * 1024 * 128 - 2)), BAD),
    (dict(k=rows(D + (1 << 40) - 8192 - 1024 + 2)), BAD),
])
def test_write_refusals(lib, kw, rc):
    s = shape()
    a = dict(l=layer(s), k=rows(), v=rows(D + 1024), slots=D, n=2)
    a.update(kw)
    assert lib.stv_kv_write(ref(s), ref(a["l"]), ref(a["k"]), ref(a["v"]), a["slots"], a["n"], None, None) == rc


# ------------------------------------------------------ stv_paged_attn ------

def call_attn(lib, s=None, spec=None, l=None, tables=D, counts=D, max_seqs=8, stride=8, seqs=D, n=2, ctx=D, row_start=D,
              max_new=1, q=None, o=None, n_rows=2, ws=D, ws_bytes=1 << 40, null=()):
    s = s or shape()
    pool = stv.stv_page_pool(None, tables, counts, 8, max_seqs, stride)
    a = {"spec": spec or stv.make_attn(), "l": l or layer(s), "pool": pool,
         "q": q or rows(heads=24, row=24 * 128), "o": o or rows(D + (1 << 30), heads=24, row=24 * 128)}
    for k in null:
        a[k] = None
    return lib.stv_paged_attn(ref(s), ref(a["spec"]), ref(a["l"]), ref(a["pool"]), seqs, n, ctx, row_start, max_new,
                              ref(a["q"]), ref(a["o"]), n_rows, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0), OK), (dict(n_rows=0), OK),
    (dict(null=("spec",)), BAD), (dict(null=("l",)), BAD), (dict(null=("pool",)), BAD), (dict(null=("q",)), BAD),
    (dict(null=("o",)), BAD), (dict(tables=None), BAD), (dict(counts=None), BAD), (dict(ctx=None), BAD),
    (dict(ws=None), BAD), (dict(ws=D + 8), BAD), (dict(n=-1), BAD), (dict(n_rows=-1), BAD), (dict(max_new=0), BAD),
    (dict(max_seqs=0), BAD), (dict(stride=0), BAD), (dict(n=4097), SHAPE), (dict(n_rows=(1 << 29) + 1), SHAPE),
    (dict(row_start=None, n=3), BAD),                       # one row each, but fewer rows
    (dict(spec=stv.make_attn(window=-1)), BAD), (dict(spec=stv.make_attn(window=1, sinks=-1)), BAD),
    (dict(spec=stv.stv_attn_spec(0, 0, 2, 0.0)), BAD), (dict(spec=stv.make_attn(scale=-1.0)), BAD),
    (dict(spec=stv.make_attn(scale=float("nan"))), BAD), (dict(spec=stv.make_attn(scale=float("inf"))), BAD),
    (dict(q=rows(heads=23, row=24 * 128)), BAD), (dict(o=rows(heads=25, row=4096)), BAD),
    (dict(q=rows(D + 1, heads=24, row=24 * 128)), BAD), (dict(q=rows(heads=24, row=128)), BAD),
    (dict(o=rows(D, heads=24, row=24 * 128)), BAD),         # over q
    (dict(o=rows(D + 256, heads=24, row=24 * 128)), BAD),   # partly
    (dict(o=rows(D + (1 << 40), heads=24, row=24 * 128)), BAD),  # in the cache
    (dict(s=shape(hd=80)), SHAPE), (dict(s=stv.make_shape()), SHAPE),
])
def test_attention_refusals(lib, kw, rc):
    assert call_attn(lib, **kw) == rc


def test_attention_workspace_refusals(lib):
    out = ctypes.c_size_t()
    s = shape()
    assert lib.stv_paged_attn_workspace_bytes(ref(s), 0, ctypes.byref(out)) == BAD
    assert lib.stv_paged_attn_workspace_bytes(ref(s), 1, None) == BAD
    assert lib.stv_paged_attn_workspace_bytes(ref(shape(hd=80)), 1, ctypes.byref(out)) == SHAPE


# ----------------------------------------------- stv_tree_accept_probs ------

@pytest.mark.parametrize("kw,rc", [
    (dict(n=0), OK), (dict(n=-1), BAD), (dict(dtype=3), BAD), (dict(drafts=2), BAD), (dict(drafts=-1), BAD),
    (dict(vocab=0), SHAPE), (dict(vocab=524289, p_stride=1 << 20, q_stride=1 << 20), SHAPE), (dict(t=0), SHAPE),
    (dict(t=33), SHAPE), (dict(parent=None), BAD), (dict(ids=None), BAD), (dict(p=None), BAD), (dict(u=None), BAD),
    (dict(n_commit=None), BAD), (dict(path=None), BAD), (dict(out=None), BAD), (dict(p_stride=999), BAD),
    (dict(q_stride=999), BAD), (dict(p=D + 2), BAD), (dict(q=D + 1), BAD), (dict(p_stride=1 << 47), BAD),
])
def test_accept_refusals(lib, kw, rc):
    a = dict(parent=D, ids=D, p=D, p_stride=1000, q=D, q_stride=1000, dtype=0, vocab=1000, drafts=0, u=D, t=8, n=2,
             n_commit=D, path=D, out=D)
    a.update(kw)
    assert lib.stv_tree_accept_probs(a["parent"], a["ids"], a["p"], a["p_stride"], a["q"], a["q_stride"], a["dtype"],
                                     a["vocab"], a["drafts"], a["u"], a["t"], a["n"], a["n_commit"], a["path"],
                                     a["out"], None, None) == rc


# ------------------------------------------------------------- Python -------

def test_python_checks():
    with pytest.raises(TypeError):
        stv.make_row_shape(8, 2, 64, torch.float32)
    with pytest.raises(ValueError):
        stv.RowCache(torch.zeros((2, 2, 2, 128, 64), dtype=BF16))
    with pytest.raises(TypeError):
        stv.RowCache(torch.zeros((2, 2, 2, 256, 64)))
    cpu = torch.zeros((4, 8))
    i = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        stv.stv_tree_accept_probs(i, i, cpu, None, torch.zeros((1, 4)), i, i, i)
    with pytest.raises(TypeError):
        stv.stv_kv_write(stv.make_row_shape(2, 2, 64, BF16), stv.RowCache(torch.zeros((2, 2, 2, 256, 64), dtype=BF16)),
                         torch.zeros((3, 2, 64), dtype=BF16), torch.zeros((3, 2, 64), dtype=BF16), i)
