"""Host-side refusals of stv_rope, stv_sample and the page calls: every
argument is checked before anything is enqueued, so they need no GPU.  Device
addresses are dummies and never dereferenced."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import opkit
import speculative_tree_verify_bit_gb300 as stv
from speculative_tree_verify_bit_gb300 import build as stv_build

D = 0x7f0000000000  # a dummy device address, 16-byte aligned
BAD, SHAPE, SMALL = stv.STV_ERR_INVALID_ARG, stv.STV_ERR_SHAPE_UNSUPPORTED, stv.STV_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    stv_build.build()
    return stv.load()


# ---------------------------------------------------------------- stv_rope --

def call_rope(lib, spec=None, dtype=1, hd=256, pos=D, n=0, q=None, qo=None, k=None, ko=None):
    spec = spec or stv.make_rope(64, (12, 10, 10))
    ref = lambda v: None if v is None else ctypes.byref(v)
    return lib.stv_rope(ctypes.byref(spec), dtype, hd, pos, n, ref(q), ref(qo), ref(k), ref(ko), 0, None)


def rows(data=D, row=1024, head=256, heads=4):
    return stv.stv_rows(data, row, head, heads)


def test_rope_no_rows_is_a_no_op(lib):
    assert call_rope(lib, q=rows(), qo=rows(D + 4096), n=0) == stv.STV_OK


@pytest.mark.parametrize("spec,rc", [
    (stv.make_rope(64, (12, 10, 10)), stv.STV_OK),
    (stv.make_rope(64, (32,)), stv.STV_OK),
    (stv.make_rope(64, (0, 32)), stv.STV_OK),
    (stv.make_rope(64, (12, 10, 9)), BAD),          # not rotary_dim / 2 pairs
    (stv.make_rope(64, (42, -10)), BAD),
    (stv.make_rope(63, (12, 10, 9)), SHAPE),        # odd
    (stv.make_rope(0, (0,)), SHAPE),
    (stv.make_rope(258, (129,)), SHAPE),            # past head_dim
    (stv.make_rope(64, (32,), theta=0.5), BAD),
    (stv.make_rope(64, (32,), theta=float("nan")), BAD),
    (stv.make_rope(64, (32,), theta=float("inf")), BAD),
    (stv.make_rope(64, (12, 10, 10), interleaved=True), stv.STV_OK),
    (stv.make_rope(64, (8, 12, 12), interleaved=True), BAD),  # axis 1's last pair would be 34
    (stv.stv_rope_spec(64, 5, (ctypes.c_int32 * 4)(32, 0, 0, 0), 0, 1e4), SHAPE),
    (stv.stv_rope_spec(64, 1, (ctypes.c_int32 * 4)(32, 0, 0, 0), 2, 1e4), BAD),
])
def test_rope_spec(lib, spec, rc):
    assert call_rope(lib, spec, q=rows(), qo=rows()) == rc


def test_rope_spec_axes_agree_with_the_plain_form(lib):
    """Interleaved sections that are accepted give every axis its pairs."""
    for sec in ((12, 10, 10), (11, 11, 10), (20, 6, 6), (16, 16), (26, 2, 2, 2)):
        spec = stv.make_rope(2 * sum(sec), sec, interleaved=True)
        assert call_rope(lib, spec, q=rows(), qo=rows()) == stv.STV_OK, sec
        assert np.bincount(opkit.pair_axes(sec, sum(sec), True), minlength=len(sec)).tolist() == list(sec)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None, qo=None), BAD),
    (dict(q=rows(), qo=None), BAD),
    (dict(q=rows(), qo=rows(), k=rows()), BAD),
    (dict(q=rows(), qo=rows(), dtype=3), BAD),
    (dict(q=rows(), qo=rows(), hd=255), SHAPE),
    (dict(q=rows(), qo=rows(), hd=514), SHAPE),
    (dict(q=rows(), qo=rows(), n=-1), BAD),
    (dict(q=rows(), qo=rows(), pos=None, n=1), BAD),
    (dict(q=rows(0), qo=rows(), n=1), BAD),
    (dict(q=rows(heads=0), qo=rows(heads=0), n=1), BAD),
    (dict(q=rows(heads=3), qo=rows(heads=4), n=1), BAD),
    (dict(q=rows(head=128), qo=rows(), n=1), BAD),            # heads overlap
    (dict(q=rows(row=512), qo=rows(), n=2), BAD),             # rows overlap
    (dict(q=rows(D + 1), qo=rows(D + 1), n=1), BAD),          # not aligned to the type
    (dict(q=rows(), qo=rows(D + 64), n=2), BAD),              # partial overlap
    (dict(q=rows(), qo=rows(row=2048), n=2), BAD),            # same data, other strides
    (dict(q=rows(), qo=rows(D + 1 << 30), k=rows(D + (1 << 20)), ko=rows(), n=2), BAD),  # k_out over q
    (dict(q=rows(), qo=rows(D + (1 << 20)), k=rows(D + (2 << 20)), ko=rows(D + (1 << 20)), n=2), BAD),  # q_out, k_out
    (dict(q=rows(row=4096, head=768), qo=rows(row=4096, head=768), k=rows(D + 256, 4096, 768),
          ko=rows(D + 256, 4096, 768), n=2), BAD),                # k's heads begin inside q's
    (dict(q=rows(row=4096, head=768), qo=rows(row=4096, head=768), k=rows(D + 1300, 4096, 768),
          ko=rows(D + 1300, 4096, 768), n=1), BAD),               # and end inside q's next ones
    (dict(q=rows(row=4096, head=768), qo=rows(row=4096, head=768), k=rows(D + 512, 4096, 512),
          ko=rows(D + 512, 4096, 512), n=2), BAD),                # head strides that differ
    (dict(q=rows(row=4096, head=768), qo=rows(row=4096, head=768), k=rows(D + 512, 4112, 768),
          ko=rows(D + 512, 4112, 768), n=2), BAD),                # row strides that differ
    (dict(q=rows(row=3100, head=768), qo=rows(row=3100, head=768), k=rows(D + 2 * 2900, 3100, 256, 1),
          ko=rows(D + 2 * 2900, 3100, 256, 1), n=3), BAD),        # k's head reaches q's next row
    (dict(q=rows(row=1 << 46), qo=rows(row=1 << 46), n=1 << 20), BAD),  # offsets past 2^48
])
def test_rope_refusals(lib, kw, rc):
    assert call_rope(lib, **kw) == rc


# -------------------------------------------------------------- stv_sample --

def call_sample(lib, logits=D, dtype=0, stride=1000, n=2, vocab=1000, rpp=1, u=D, ids=D):
    return lib.stv_sample(logits, dtype, stride, n, vocab, None, None, None, None, rpp, u, ids, None, None, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0), stv.STV_OK),
    (dict(n=-1), BAD),
    (dict(vocab=0), BAD),
    (dict(vocab=(1 << 19) + 1, stride=1 << 20), SHAPE),
    (dict(stride=999), BAD),
    (dict(rpp=0), BAD),
    (dict(dtype=3), BAD),
    (dict(logits=None), BAD),
    (dict(u=None), BAD),
    (dict(ids=None), BAD),
    (dict(logits=D + 2), BAD),
    (dict(logits=D + 1, dtype=2), BAD),
])
def test_sample_refusals(lib, kw, rc):
    assert call_sample(lib, **kw) == rc


# ------------------------------------------------------------------- pages --

def pool(refs=D, tables=D, counts=D, n_pages=100, max_seqs=8, stride=20):
    return stv.stv_page_pool(refs, tables, counts, n_pages, max_seqs, stride)


@pytest.mark.parametrize("p,rc", [
    (pool(), stv.STV_OK),
    (pool(refs=None), BAD), (pool(tables=None), BAD), (pool(counts=None), BAD),
    (pool(n_pages=0), BAD), (pool(max_seqs=0), BAD), (pool(stride=0), BAD),
    (pool(n_pages=262145), SHAPE), (pool(max_seqs=4097), SHAPE),
    (pool(n_pages=262144, max_seqs=4096), stv.STV_OK),
])
def test_pool_checks(lib, p, rc):
    assert lib.stv_page_reserve(ctypes.byref(p), D, 0, D, 16, None, None) == rc
    assert lib.stv_page_free(ctypes.byref(p), D, 0, None, None) == rc


@pytest.mark.parametrize("n,rc", [(1, stv.STV_OK), (100, stv.STV_OK), (262144, stv.STV_OK), (0, BAD), (-5, BAD),
                                  (262145, SHAPE)])
def test_page_workspace(lib, n, rc):
    out = ctypes.c_size_t()
    assert lib.stv_page_workspace_bytes(n, ctypes.byref(out)) == rc
    assert rc != stv.STV_OK or out.value == 16 + 8 * n
    assert lib.stv_page_workspace_bytes(n, None) != stv.STV_OK


def test_page_list_checks(lib):
    p = ctypes.byref(pool())
    assert lib.stv_page_reserve(p, D, 9, D, 16, None, None) == BAD      # more than max_seqs
    assert lib.stv_page_reserve(p, D, -1, D, 16, None, None) == BAD
    assert lib.stv_page_reserve(p, D, 2, D, -1, None, None) == BAD
    assert lib.stv_page_reserve(p, None, 2, D, 16, None, None) == BAD
    assert lib.stv_page_reserve(p, D, 2, None, 16, None, None) == BAD
    assert lib.stv_page_free(p, D, 9, None, None) == BAD
    assert lib.stv_page_free(p, None, 1, None, None) == BAD


def layers(n=2, n_pages=100, page_bytes=229376, data=D):
    return (stv.stv_layer_cache * max(n, 1))(*[stv.stv_layer_cache(data, page_bytes, n_pages)] * max(n, 1))


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0), stv.STV_OK),
    (dict(n=9), BAD), (dict(n=-1), BAD), (dict(src=None, n=1), BAD), (dict(dst=None, n=1), BAD),
    (dict(ctx=None, n=1), BAD),
    (dict(n_layers=0), BAD), (dict(n_layers=129), BAD),
    (dict(lay=layers(n_pages=99)), BAD),                # a pool shorter than the books
    (dict(lay=layers(page_bytes=57344)), SHAPE),        # not this shape's pages
    (dict(lay=layers(data=D + 8)), BAD),
    (dict(ws=None), BAD), (dict(ws=D + 8), BAD), (dict(ws_bytes=815), SMALL),
])
def test_fork_compact_copy_refusals(lib, kw, rc):
    a = dict(n=0, n_layers=2, lay=layers(), src=D, dst=D, ctx=D, ws=D, ws_bytes=816)
    a.update(kw)
    sh, p = stv.make_shape(), pool()
    assert lib.stv_page_fork(ctypes.byref(sh), a["lay"], a["n_layers"], ctypes.byref(p), a["src"], a["dst"], a["n"],
                             a["ctx"], a["ws"], a["ws_bytes"], None, None) == rc
    if "ctx" not in kw and kw.get("n") != 9:
        assert lib.stv_page_copy(ctypes.byref(sh), a["lay"], a["n_layers"], 100, a["src"], a["dst"], a["n"], a["ws"],
                                 a["ws_bytes"], None, None) == rc
    if not {"n", "src", "dst", "ctx"} & set(kw):
        assert lib.stv_page_compact(ctypes.byref(sh), a["lay"], a["n_layers"], ctypes.byref(p), D, D, a["ws"],
                                    a["ws_bytes"], None, None) == rc


def test_compact_needs_its_outputs(lib):
    sh, p, lay = stv.make_shape(), pool(), layers()
    for m, n in ((None, D), (D, None)):
        assert lib.stv_page_compact(ctypes.byref(sh), lay, 2, ctypes.byref(p), m, n, D, 816, None, None) == BAD


def test_layers_are_looked_over_in_every_call():
    """A pool that is given another tensor at the same address between two
    calls (CPU tensors: device -1)."""
    storage = torch.zeros(2 * 2 * 57344, dtype=torch.uint8)
    layer = stv.LayerCache(storage[:2 * 57344], 1)
    want = struct.pack("@Pqi4x", storage.data_ptr(), 57344, 2)
    assert stv._layer_array([layer], -1) == want
    layer.pool = storage[::2]
    with pytest.raises(ValueError):
        stv._layer_array([layer], -1)
    layer.pool = storage[:2 * 57344]
    assert stv._layer_array([layer, layer], -1) == 2 * want
    with pytest.raises(ValueError):
        stv._layer_array([layer], 0)


# ---------------------------------------------- the plain forms themselves --

def test_plain_sample_against_counts():
    """Every token is drawn for exactly its share of evenly spaced u."""
    x = np.array([1.0, -np.inf, 2.0, 2.0, 0.0])
    n = 4000
    got = np.bincount([opkit.sample(x, (i + 0.5) / n, t=0.5)[0] for i in range(n)], minlength=5) / n
    w = np.where(np.isfinite(x), np.exp(2 * x), 0)
    assert np.abs(got - w / w.sum()).max() <= 1.0 / n
    assert opkit.sample(x, 0.9, top_k=1)[0] == 2          # a tie: the lower index
    assert opkit.sample(x, 0.99, top_p=0.3)[0] == 2
    assert {opkit.sample(x, v, min_p=0.99)[0] for v in (0.1, 0.4, 0.6, 0.9)} == {2, 3}


def test_plain_rope_is_a_rotation():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 16))
    pos = rng.integers(0, 300000, (3, 5))
    y = opkit.rope(x, pos, 12, (2, 2, 2), 1e4, True)
    assert np.allclose(opkit.rope(y, pos, 12, (2, 2, 2), 1e4, True, inverse=True), x, atol=1e-12)
    assert np.array_equal(y[..., 12:], x[..., 12:])


def test_plain_books_stay_consistent():
    b = opkit.Books(40, 6, 12)
    b.ctx[:2] = 700, 256
    b.reserve([0, 1], 16)
    b.fork([0, 0, 1], [2, 3, 4])
    b.reserve([2, 3, 4], 16)
    b.free([0])
    where, n = b.compact()
    held = np.bincount(b.tables[b.tables >= 0], minlength=40)
    assert np.array_equal(held, b.refs) and n == np.count_nonzero(b.refs) and (b.refs[:n] > 0).all()
