"""Python binding of libstv.so -- the GB300 (sm_103a) tree-verify library.

Argument marshalling only: every function has the name of the C entry point
it calls (include/stv.h), takes torch CUDA tensors for the device pointers
and raises ``StvError`` on a negative status.  Every step of the round runs
in the library's CUDA kernels; there is no other implementation behind these
names, and importing a function fails loudly when the library is not built
(``python -m speculative_tree_verify_bit_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libstv.so")

STV_OK = 0
STV_ERR_INVALID_ARG = -1
STV_ERR_SHAPE_UNSUPPORTED = -2
STV_ERR_WORKSPACE_TOO_SMALL = -3
STV_ERR_CUDA = -4
STV_ERR_UNIMPLEMENTED = -5

STV_DEV_BAD_PAGE = 1
STV_DEV_BAD_TREE = 2
STV_DEV_BAD_ROW = 4
STV_DEV_BAD_COMMIT = 8
STV_DEV_TIMEOUT = 16
STV_DEV_BAD_SAMPLE = 32
STV_DEV_NO_PAGES = 64
STV_DEV_BAD_SEQ = 128

STV_KV_BY_GROUP = 0  # group 32: the 3-bit cache; group 256: the int4 per-token-head cache
STV_KV_K4V2 = 2      # the K 4 / V 2-bit cache (group 32)
STV_KV_ROWS_F16 = 4  # the drafter's cache: rows as they are (group 0)
STV_KV_ROWS_BF16 = 5

STV_PATH_EXACT = 0
STV_PATH_INT8 = 1
PATHS = {"exact": STV_PATH_EXACT, "int8": STV_PATH_INT8}

STV_MAX_SEQS = 64
HEAD_DIM = 256
GROUP = 32
PAGE_TOKENS = 256
HEAD_BLOCK_BYTES = 57344
GROUP_INT4 = 256                # the int4 per-token-head cache (include/stv.h)
HEAD_BLOCK_BYTES_INT4 = 66560

# Every symbol include/stv.h declares.
EXPORTS = (
    "stv_status_string", "stv_version", "stv_page_bytes", "stv_kv_append_pack", "stv_verify_workspace_bytes",
    "stv_verify_attn", "stv_split_combine", "stv_tree_accept", "stv_kv_commit", "stv_int8_qk_dots",
    "stv_verify_attn_no_alloc", "stv_append_verify_attn", "stv_lookup_workspace_bytes", "stv_lookup_draft",
    "stv_prefill_workspace_bytes", "stv_prefill_attn", "stv_verify_attn_timeout_test",
    "stv_prefill_attn_timeout_test", "stv_append_verify_combine", "stv_rope", "stv_sample",
    "stv_page_workspace_bytes", "stv_page_reserve", "stv_page_fork", "stv_page_free", "stv_page_compact",
    "stv_page_copy", "stv_page_extend", "stv_kv_write", "stv_paged_attn_workspace_bytes", "stv_paged_attn",
    "stv_tree_accept_probs", "stv_paged_attn_timeout_test",
)


class StvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


class stv_shape(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("kv_format", ctypes.c_int32)]


class stv_layer_cache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("n_pages", ctypes.c_int32)]


class stv_history(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("n", ctypes.c_int64)]


class stv_seq(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("ctx", ctypes.c_int32)]


class stv_rope_spec(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("interleaved", ctypes.c_int32), ("theta", ctypes.c_double)]


class stv_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class stv_attn_spec(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class stv_page_pool(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("tables", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("max_seqs", ctypes.c_int32), ("table_stride", ctypes.c_int32)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libstv.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m speculative_tree_verify_bit_gb300.build` (no fallback exists)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, I32, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_int64
        lib.stv_status_string.restype = ctypes.c_char_p
        lib.stv_status_string.argtypes = [I]
        lib.stv_version.restype = I
        lib.stv_page_bytes.restype = I
        lib.stv_page_bytes.argtypes = [P, P]
        lib.stv_kv_append_pack.restype = I
        lib.stv_kv_append_pack.argtypes = [P, P, P, I, P, P, P, P, I, P, P]
        lib.stv_verify_workspace_bytes.restype = I
        lib.stv_verify_workspace_bytes.argtypes = [P, P, I, I, I, P]
        lib.stv_verify_attn.restype = I
        lib.stv_verify_attn.argtypes = [P, P, P, I, P, P, I, I, P, ctypes.c_size_t, P, P]
        lib.stv_split_combine.restype = I
        lib.stv_split_combine.argtypes = [P, P, I, I, P, ctypes.c_size_t, P, P]
        lib.stv_tree_accept.restype = I
        lib.stv_tree_accept.argtypes = [P, P, P, I, I, P, P, P, P, P]
        lib.stv_kv_commit.restype = I
        lib.stv_kv_commit.argtypes = [P, P, I, P, I, I, P, P, P, P, P]
        lib.stv_int8_qk_dots.restype = I
        lib.stv_int8_qk_dots.argtypes = [P, P, P, P, P, I, P, ctypes.c_size_t, P, P, P]
        lib.stv_prefill_workspace_bytes.restype = I
        lib.stv_prefill_workspace_bytes.argtypes = [P, P, I, P]
        lib.stv_prefill_attn.restype = I
        lib.stv_prefill_attn.argtypes = [P, P, P, P, I, I, P, ctypes.c_size_t, P, P, P]
        lib.stv_lookup_workspace_bytes.restype = I
        lib.stv_lookup_workspace_bytes.argtypes = [I, P]
        lib.stv_lookup_draft.restype = I
        lib.stv_lookup_draft.argtypes = [P, I, I, I, I, P, P, P, P, P, ctypes.c_size_t, P]
        lib.stv_append_verify_attn.restype = I
        lib.stv_append_verify_attn.argtypes = [P, P, P, I, P, P, P, P, I, I, P, ctypes.c_size_t, P, P]
        lib.stv_append_verify_combine.restype = I
        lib.stv_append_verify_combine.argtypes = [P, P, P, I, P, P, P, P, I, I, P, ctypes.c_size_t, P, P, P]
        lib.stv_verify_attn_no_alloc.restype = I
        lib.stv_verify_attn_no_alloc.argtypes = [P, P, P, I, P, P, I, I, P, P, P]
        lib.stv_verify_attn_timeout_test.restype = I
        lib.stv_verify_attn_timeout_test.argtypes = [P, P, P, I, P, P, I, I, P, ctypes.c_size_t, P, P]
        lib.stv_rope.restype = I
        lib.stv_rope.argtypes = [P, I, I, P, I, P, P, P, P, I, P]
        lib.stv_sample.restype = I
        lib.stv_sample.argtypes = [P, I, I64, I, I, P, P, P, P, I, P, P, P, P, P]
        lib.stv_page_workspace_bytes.restype = I
        lib.stv_page_workspace_bytes.argtypes = [I, P]
        lib.stv_page_reserve.restype = I
        lib.stv_page_reserve.argtypes = [P, P, I, P, I, P, P]
        lib.stv_page_fork.restype = I
        lib.stv_page_fork.argtypes = [P, P, I, P, P, P, I, P, P, ctypes.c_size_t, P, P]
        lib.stv_page_free.restype = I
        lib.stv_page_free.argtypes = [P, P, I, P, P]
        lib.stv_page_compact.restype = I
        lib.stv_page_compact.argtypes = [P, P, I, P, P, P, P, ctypes.c_size_t, P, P]
        lib.stv_page_copy.restype = I
        lib.stv_page_copy.argtypes = [P, P, I, I, P, P, I, P, ctypes.c_size_t, P, P]
        lib.stv_page_extend.restype = I
        lib.stv_page_extend.argtypes = [P, P, I, P, P, P, P, P, P, I, P, P]
        lib.stv_kv_write.restype = I
        lib.stv_kv_write.argtypes = [P, P, P, P, P, I, P, P]
        lib.stv_paged_attn_workspace_bytes.restype = I
        lib.stv_paged_attn_workspace_bytes.argtypes = [P, I, P]
        lib.stv_paged_attn.restype = I
        lib.stv_paged_attn.argtypes = [P, P, P, P, P, I, P, P, I, P, P, I, P, ctypes.c_size_t, P, P]
        lib.stv_paged_attn_timeout_test.restype = I
        lib.stv_paged_attn_timeout_test.argtypes = lib.stv_paged_attn.argtypes
        lib.stv_tree_accept_probs.restype = I
        lib.stv_tree_accept_probs.argtypes = [P, P, P, I64, P, I64, I, I, I, P, I, I, P, P, P, P, P]
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().stv_status_string(int(status)).decode()


def _check(fn: str, rc: int):
    if rc != STV_OK:
        raise StvError(fn, rc)


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------

def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    import torch

    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_shape(hq: int = 24, hkv: int = 4, group: int = GROUP, kv_format: int = STV_KV_BY_GROUP) -> stv_shape:
    """group 32: the 3-bit cache; group 256 (GROUP_INT4): the int4
    per-token-head cache; kv_format STV_KV_K4V2 (group 32): the K 4 / V 2-bit
    cache (include/stv.h)."""
    return stv_shape(hq, hkv, HEAD_DIM, group, PAGE_TOKENS, kv_format)


def head_block_bytes(group: int = GROUP) -> int:
    return HEAD_BLOCK_BYTES_INT4 if group == GROUP_INT4 else HEAD_BLOCK_BYTES


class LayerCache:
    """One layer's paged pool: a uint8 CUDA tensor of n_pages * page_bytes."""

    def __init__(self, pool, hkv: int, group: int = GROUP):
        import torch

        self.hkv = hkv
        self.group = group
        self.page_bytes = hkv * head_block_bytes(group)
        assert pool.dtype == torch.uint8 and pool.numel() % self.page_bytes == 0
        self.pool = pool
        self.n_pages = pool.numel() // self.page_bytes

    @classmethod
    def empty(cls, n_pages: int, hkv: int = 4, device="cuda", group: int = GROUP):
        import torch

        return cls(torch.zeros(n_pages * hkv * head_block_bytes(group), dtype=torch.uint8, device=device), hkv, group)

    def c(self) -> stv_layer_cache:
        return stv_layer_cache(_ptr(self.pool, name="pool").value, self.page_bytes, self.n_pages)


class Seq:
    """A sequence: its device page table (int32) and its context length."""

    def __init__(self, page_table, ctx: int):
        self.page_table = page_table
        self.ctx = int(ctx)

    def c(self) -> stv_seq:
        import torch

        return stv_seq(_ptr(self.page_table, torch.int32, "page_table").value, self.page_table.numel(), self.ctx)


def _seq_array(seqs):
    arr = (stv_seq * len(seqs))()
    for i, s in enumerate(seqs):
        arr[i] = s.c()
    return arr


# --------------------------------------------------------------------------
# entry points (same names as include/stv.h)
# --------------------------------------------------------------------------

def stv_version() -> int:
    return load().stv_version()


def stv_page_bytes(shape: stv_shape) -> int:
    out = ctypes.c_int64()
    _check("stv_page_bytes", load().stv_page_bytes(ctypes.byref(shape), ctypes.byref(out)))
    return out.value


def stv_kv_append_pack(shape, layer: LayerCache, seqs, k, v, row_seq, row_pos, dev_status=None, stream=None):
    import torch

    lc = layer.c()
    arr = _seq_array(seqs)
    _check("stv_kv_append_pack", load().stv_kv_append_pack(
        ctypes.byref(shape), ctypes.byref(lc), arr, len(seqs), _ptr(k, torch.float16, "k"), _ptr(v, torch.float16, "v"),
        _ptr(row_seq, torch.int32, "row_seq"), _ptr(row_pos, torch.int32, "row_pos"), row_seq.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_verify_workspace_bytes(shape, seqs, t_nodes: int, sm_count: int = 0) -> int:
    out = ctypes.c_size_t()
    arr = _seq_array(seqs)
    _check("stv_verify_workspace_bytes", load().stv_verify_workspace_bytes(
        ctypes.byref(shape), arr, len(seqs), int(t_nodes), int(sm_count), ctypes.byref(out)))
    return out.value


def stv_verify_attn(shape, layer: LayerCache, seqs, q, parent, t_nodes: int, path, workspace, dev_status=None,
                    stream=None):
    import torch

    lc = layer.c()
    arr = _seq_array(seqs)
    path = PATHS.get(path, path)
    _check("stv_verify_attn", load().stv_verify_attn(
        ctypes.byref(shape), ctypes.byref(lc), arr, len(seqs), _ptr(q, torch.float16, "q"),
        _ptr(parent, torch.int32, "parent"), int(t_nodes), int(path), _ptr(workspace, name="workspace"),
        workspace.numel() * workspace.element_size(), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_append_verify_attn(shape, layer: LayerCache, seqs, k_tree, v_tree, q, parent, t_nodes: int, path, workspace,
                           dev_status=None, stream=None):
    """stv_kv_append_pack of the round's tree rows (k_tree, v_tree: fp16
    [n_seqs][T][hkv][256], row i of sequence s at ctx_s + i) fused into
    stv_verify_attn: one launch.  The workspace must be zero-filled before
    its first use here (arrival counters of the exact path's packing warp);
    each completed call leaves them zero."""
    import torch

    lc = layer.c()
    arr = _seq_array(seqs)
    path = PATHS.get(path, path)
    _check("stv_append_verify_attn", load().stv_append_verify_attn(
        ctypes.byref(shape), ctypes.byref(lc), arr, len(seqs), _ptr(k_tree, torch.float16, "k_tree"),
        _ptr(v_tree, torch.float16, "v_tree"), _ptr(q, torch.float16, "q"), _ptr(parent, torch.int32, "parent"),
        int(t_nodes), int(path), _ptr(workspace, name="workspace"), workspace.numel() * workspace.element_size(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_append_verify_combine(shape, layer: LayerCache, seqs, k_tree, v_tree, q, parent, t_nodes: int, path,
                              workspace, o, dev_status=None, stream=None):
    """stv_kv_append_pack of the round's tree rows + stv_verify_attn +
    stv_split_combine in one cooperative launch.  The workspace (the size
    stv_verify_workspace_bytes gives) must be zero-filled before its first
    use here; each completed call leaves its counters zero."""
    import torch

    lc = layer.c()
    arr = _seq_array(seqs)
    path = PATHS.get(path, path)
    _check("stv_append_verify_combine", load().stv_append_verify_combine(
        ctypes.byref(shape), ctypes.byref(lc), arr, len(seqs), _ptr(k_tree, torch.float16, "k_tree"),
        _ptr(v_tree, torch.float16, "v_tree"), _ptr(q, torch.float16, "q"), _ptr(parent, torch.int32, "parent"),
        int(t_nodes), int(path), _ptr(workspace, name="workspace"), workspace.numel() * workspace.element_size(),
        _ptr(o, torch.float16, "o"), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_split_combine(shape, seqs, t_nodes: int, workspace, o, stream=None):
    import torch

    arr = _seq_array(seqs)
    _check("stv_split_combine", load().stv_split_combine(
        ctypes.byref(shape), arr, len(seqs), int(t_nodes), _ptr(workspace, name="workspace"),
        workspace.numel() * workspace.element_size(), _ptr(o, torch.float16, "o"), _stream(stream)))


def stv_tree_accept(parent, draft_ids, target_argmax, n_commit, path, out_ids, dev_status=None, stream=None):
    import torch

    n_seqs, t = parent.shape
    _check("stv_tree_accept", load().stv_tree_accept(
        _ptr(parent, torch.int32, "parent"), _ptr(draft_ids, torch.int32, "draft_ids"),
        _ptr(target_argmax, torch.int32, "target_argmax"), int(t), int(n_seqs), _ptr(n_commit, torch.int32, "n_commit"),
        _ptr(path, torch.int32, "path"), _ptr(out_ids, torch.int32, "out_ids"),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_kv_commit(shape, layers, seqs, t_nodes: int, n_commit, path, ctx_dev=None, dev_status=None, stream=None):
    import torch

    larr = (stv_layer_cache * len(layers))()
    for i, l in enumerate(layers):
        larr[i] = l.c()
    arr = _seq_array(seqs)
    _check("stv_kv_commit", load().stv_kv_commit(
        ctypes.byref(shape), larr, len(layers), arr, len(seqs), int(t_nodes), _ptr(n_commit, torch.int32, "n_commit"),
        _ptr(path, torch.int32, "path"), _ptr(ctx_dev, torch.int32, "ctx_dev"),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_int8_qk_dots(shape, layer: LayerCache, seq: Seq, q, parent, t_nodes: int, workspace, dots, dev_status=None,
                     stream=None):
    """The int8 verify of one sequence, also writing the kernel's own
    per-group integer dots: dots int32 [hkv][T*G][ctx+T][8]."""
    import torch

    lc = layer.c()
    arr = _seq_array([seq])
    _check("stv_int8_qk_dots", load().stv_int8_qk_dots(
        ctypes.byref(shape), ctypes.byref(lc), arr, _ptr(q, torch.float16, "q"), _ptr(parent, torch.int32, "parent"),
        int(t_nodes), _ptr(workspace, name="workspace"), workspace.numel() * workspace.element_size(),
        _ptr(dots, torch.int32, "dots"), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_verify_attn_timeout_test(shape, layer: LayerCache, seqs, q, parent, t_nodes: int, path, workspace,
                                 dev_status=None, stream=None):
    """stv_verify_attn with the kernel's copies withheld: every wait runs out
    and the kernel reports STV_DEV_TIMEOUT (failure-path test)."""
    import torch

    lc = layer.c()
    arr = _seq_array(seqs)
    path = PATHS.get(path, path)
    _check("stv_verify_attn_timeout_test", load().stv_verify_attn_timeout_test(
        ctypes.byref(shape), ctypes.byref(lc), arr, len(seqs), _ptr(q, torch.float16, "q"),
        _ptr(parent, torch.int32, "parent"), int(t_nodes), int(path), _ptr(workspace, name="workspace"),
        workspace.numel() * workspace.element_size(), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_verify_attn_no_alloc(shape, layer: LayerCache, seqs, q, parent, t_nodes: int, path, o, dev_status=None,
                             stream=None):
    """Verify attention + split merge with the library's own fixed scratch
    (for callers that cannot allocate device memory; see include/stv.h)."""
    import torch

    lc = layer.c()
    arr = _seq_array(seqs)
    path = PATHS.get(path, path)
    _check("stv_verify_attn_no_alloc", load().stv_verify_attn_no_alloc(
        ctypes.byref(shape), ctypes.byref(lc), arr, len(seqs), _ptr(q, torch.float16, "q"),
        _ptr(parent, torch.int32, "parent"), int(t_nodes), int(path), _ptr(o, torch.float16, "o"),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_lookup_workspace_bytes(n_seqs: int) -> int:
    out = ctypes.c_size_t()
    _check("stv_lookup_workspace_bytes", load().stv_lookup_workspace_bytes(int(n_seqs), ctypes.byref(out)))
    return out.value


def stv_lookup_draft(histories, min_len: int, max_len: int, k: int, n_prop, prop, match_len, match_pos, workspace,
                     stream=None):
    """Lookup drafting over each history (int32 CUDA tensors): the up to k
    tokens that followed the latest earlier occurrence of the longest suffix
    of length max_len .. min_len (include/stv.h).  The workspace must be zero
    before its first use; each call leaves it zero."""
    import torch

    arr = (stv_history * len(histories))()
    for i, t in enumerate(histories):
        arr[i].tokens = _ptr(t, torch.int32, "history").value if t.numel() else None
        arr[i].n = t.numel()
    _check("stv_lookup_draft", load().stv_lookup_draft(
        arr, len(histories), int(min_len), int(max_len), int(k), _ptr(n_prop, torch.int32, "n_prop"),
        _ptr(prop, torch.int32, "prop"), _ptr(match_len, torch.int32, "match_len"),
        _ptr(match_pos, torch.int64, "match_pos"), _ptr(workspace, name="workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def stv_prefill_workspace_bytes(shape, seq, n_tokens: int) -> int:
    arr = _seq_array([seq])
    out = ctypes.c_size_t()
    _check("stv_prefill_workspace_bytes", load().stv_prefill_workspace_bytes(
        ctypes.byref(shape), arr, int(n_tokens), ctypes.byref(out)))
    return out.value


def stv_prefill_attn(shape, layer: LayerCache, seq, q, n_tokens: int, path, workspace, o, dev_status=None,
                     stream=None):
    """Prefill attention over the 3-bit cache (include/stv.h): q and o are
    fp16 [n_tokens][hq][256]; the prompt's rows are already in the cache at
    seq.ctx .. seq.ctx + n_tokens - 1."""
    import torch

    lc = layer.c()
    arr = _seq_array([seq])
    path = PATHS.get(path, path)
    _check("stv_prefill_attn", load().stv_prefill_attn(
        ctypes.byref(shape), ctypes.byref(lc), arr, _ptr(q, torch.float16, "q"), int(n_tokens), int(path),
        _ptr(workspace, name="workspace"), workspace.numel() * workspace.element_size(),
        _ptr(o, torch.float16, "o"), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def stv_prefill_attn_timeout_test(shape, layer: LayerCache, seq, q, n_tokens: int, path, workspace, o,
                                  dev_status=None, stream=None):
    """stv_prefill_attn with the persistent kernel's copies withheld: every
    wait runs out and the kernel reports STV_DEV_TIMEOUT (failure-path test)."""
    import torch

    lc = layer.c()
    arr = _seq_array([seq])
    path = PATHS.get(path, path)
    _check("stv_prefill_attn_timeout_test", load().stv_prefill_attn_timeout_test(
        ctypes.byref(shape), ctypes.byref(lc), arr, _ptr(q, torch.float16, "q"), int(n_tokens), int(path),
        _ptr(workspace, name="workspace"), workspace.numel() * workspace.element_size(),
        _ptr(o, torch.float16, "o"), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


# --------------------------------------------------------------------------
# around the round: rotary positions, sampling, the pages of the caches
# --------------------------------------------------------------------------

# These calls take a few microseconds on the GPU, so the marshalling is kept
# short: raw pointers and packed structs, torch imported once.
_torch = None
_ROWS = struct.Struct("@Pqqi4x")  # stv_rows
_DTYPES = {}


def _t():
    global _torch
    if _torch is None:
        import torch

        _DTYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})  # enum stv_dtype
        _torch = torch
    return _torch


def _device_of(t, name):
    """The CUDA device of the call, which is the current one (the kernels are
    launched there)."""
    torch = _t()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev, cur = t.get_device(), torch.cuda.current_device()
    if dev != cur:
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{cur}")
    return dev


def _raw(t, dtype, dev, name, n=None):
    """Address of a contiguous tensor of the call's device (None: no tensor),
    of n entries where n is given."""
    if t is None:
        return None
    if not isinstance(t, _torch.Tensor) or t.get_device() != dev:
        raise (TypeError if not isinstance(t, _torch.Tensor) or not t.is_cuda else ValueError)(
            f"{name} must be a CUDA tensor on cuda:{dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    return t.data_ptr()


def _raw_stream(stream, dev):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(dtype, name):
    try:
        return _DTYPES[dtype]
    except KeyError:
        raise TypeError(f"{name} must be fp32, fp16 or bf16, got {dtype}") from None


def make_rope(rotary_dim: int, sections, theta: float = 10000.0, interleaved: bool = False) -> stv_rope_spec:
    """Rotary positions over rotary_dim channels with len(sections) axes,
    sections[a] channel pairs each (include/stv.h)."""
    if not 1 <= len(sections) <= 4:
        raise ValueError(f"1 to 4 axes, got {len(sections)}")
    sec = (ctypes.c_int32 * 4)(*[int(n) for n in sections])
    return stv_rope_spec(int(rotary_dim), len(sections), sec, int(interleaved), float(theta))


def _rows(t, n_rows, head_dim, dtype, dev, name):
    if t is None:
        return None
    if not isinstance(t, _torch.Tensor) or t.get_device() != dev:
        raise (TypeError if not isinstance(t, _torch.Tensor) or not t.is_cuda else ValueError)(
            f"{name} must be a CUDA tensor on cuda:{dev}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != n_rows or shape[2] != head_dim:
        raise ValueError(f"{name} must be [{n_rows}][heads][{head_dim}], got {list(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    row, head, last = t.stride()
    if last != 1 and head_dim > 1:
        raise ValueError(f"{name} must have adjacent channels")
    heads = shape[1]
    return _ROWS.pack(t.data_ptr(), row, head if heads > 1 or head >= head_dim else head_dim, heads)


def stv_rope(spec: stv_rope_spec, pos, q, q_out, k=None, k_out=None, inverse: bool = False, stream=None):
    """Rotary positions with several axes: q, k [n_rows][heads][head_dim]
    (fp32, fp16 or bf16; any row and head strides) turned by pos, int32
    [n_axes][n_rows], into q_out, k_out (the input itself: in place).  q or k
    may be None.  inverse: the gradient, by the opposite angles."""
    torch = _t()
    first = q if q is not None else k
    if first is None or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q with q_out, k with k_out, or both pairs")
    dev = _device_of(first, "q")
    if first.dim() != 3:
        raise ValueError("q and k must be [n_rows][heads][head_dim]")
    n, _, hd = first.shape
    dt = first.dtype
    if tuple(pos.shape) != (spec.n_axes, n):
        raise ValueError(f"pos must be [{spec.n_axes}][{n}], got {list(pos.shape)}")
    rc = load().stv_rope(
        ctypes.byref(spec), _dtype_code(dt, "q"), hd, _raw(pos, torch.int32, dev, "pos"), n,
        _rows(q, n, hd, dt, dev, "q"), _rows(q_out, n, hd, dt, dev, "q_out"), _rows(k, n, hd, dt, dev, "k"),
        _rows(k_out, n, hd, dt, dev, "k_out"), 1 if inverse else 0, _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_rope", rc)


def stv_sample(logits, u, ids, logprob=None, temperature=None, top_k=None, top_p=None, min_p=None,
               rows_per_param: int = 1, dev_status=None, stream=None):
    """One token per row of logits [n_rows][vocab] (fp32, fp16 or bf16, rows
    any distance apart), drawn with u [n_rows] in [0, 1) from the row's
    distribution under temperature, top_k, top_p and min_p, one entry of each
    for rows_per_param rows (None: 1, all, 1, 0); ids int32 [n_rows], logprob
    fp32 [n_rows] or None (include/stv.h)."""
    torch = _t()
    dev = _device_of(logits, "logits")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [n_rows][vocab] with adjacent columns")
    n, vocab = logits.shape
    rpp = int(rows_per_param)
    if rpp < 1:
        raise ValueError(f"rows_per_param must be at least 1, got {rpp}")
    m = -(-n // rpp)
    f32, i32 = torch.float32, torch.int32
    rc = load().stv_sample(
        logits.data_ptr(), _dtype_code(logits.dtype, "logits"), logits.stride(0) if n > 1 else vocab, n, vocab,
        _raw(temperature, f32, dev, "temperature", m), _raw(top_k, i32, dev, "top_k", m),
        _raw(top_p, f32, dev, "top_p", m), _raw(min_p, f32, dev, "min_p", m), rpp, _raw(u, f32, dev, "u", n),
        _raw(ids, i32, dev, "ids", n), _raw(logprob, f32, dev, "logprob", n),
        _raw(dev_status, i32, dev, "dev_status"), _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_sample", rc)


class PagePool:
    """The books of a page pool (include/stv.h): refs int32 [n_pages], tables
    int32 [max_seqs][table_stride], counts int32 [max_seqs], on the device.
    The pool holds the tensors; give it others only by making another pool."""

    def __init__(self, refs, tables, counts):
        i32 = _t().int32
        if tables.dim() != 2 or refs.dim() != 1:
            raise ValueError("refs must be [n_pages], tables [max_seqs][table_stride]")
        self._dev = dev = _device_of(refs, "refs")
        self.refs, self.tables, self.counts = refs, tables, counts
        m, stride = tables.shape
        self._c = stv_page_pool(_raw(refs, i32, dev, "refs"), _raw(tables, i32, dev, "tables"),
                                _raw(counts, i32, dev, "counts", m), refs.numel(), m, stride)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages: int, max_seqs: int, table_stride: int, device="cuda"):
        """All pages free, no sequence holding any."""
        torch = _t()
        z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)
        return cls(z(n_pages), torch.full((max_seqs, table_stride), -1, dtype=torch.int32, device=device), z(max_seqs))

    def c(self) -> stv_page_pool:
        return self._c

    def seq(self, s: int, n_pages: int, ctx: int) -> Seq:
        """Sequence s as the round's calls take it: the first n_pages of its
        table, ctx cached tokens."""
        return Seq(self.tables[s, :n_pages], ctx)

    def _on_current(self):
        cur = _t().cuda.current_device()
        if cur != self._dev:
            raise ValueError(f"the pool is on cuda:{self._dev}, but the current device is cuda:{cur}")
        return self._dev


def _layer_array(layers, dev):
    """The layers' stv_layer_cache array, packed."""
    flat = []
    for l in layers:
        pool = l.pool
        if pool.get_device() != dev or not pool.is_contiguous():
            raise ValueError(f"the layers' pools must be contiguous CUDA tensors on cuda:{dev}")
        flat += (pool.data_ptr(), l.page_bytes, l.n_pages)
    return struct.pack("@" + "Pqi4x" * len(layers), *flat)


def stv_page_workspace_bytes(pool) -> int:
    """Workspace bytes of the page calls on a PagePool, or on so many pages."""
    n = pool._c.n_pages if isinstance(pool, PagePool) else int(pool)
    out = ctypes.c_size_t()
    _check("stv_page_workspace_bytes", load().stv_page_workspace_bytes(n, ctypes.byref(out)))
    return out.value


def stv_page_reserve(pool: PagePool, seqs, ctx, extra: int, dev_status=None, stream=None):
    """Pages for ctx[s] + extra tokens for every sequence of the list (int32
    CUDA tensor); ctx int32 [max_seqs] on the device."""
    dev, i32 = pool._on_current(), _torch.int32
    rc = load().stv_page_reserve(
        pool._ref, _raw(seqs, i32, dev, "seqs"), seqs.numel(), _raw(ctx, i32, dev, "ctx", pool._c.max_seqs),
        int(extra), _raw(dev_status, i32, dev, "dev_status"), _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_page_reserve", rc)


def stv_page_free(pool: PagePool, seqs, dev_status=None, stream=None):
    """The listed sequences give up their pages."""
    dev, i32 = pool._on_current(), _torch.int32
    rc = load().stv_page_free(pool._ref, _raw(seqs, i32, dev, "seqs"), seqs.numel(),
                              _raw(dev_status, i32, dev, "dev_status"), _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_page_free", rc)


def stv_page_fork(shape, layers, pool: PagePool, src, dst, ctx, workspace, dev_status=None, stream=None):
    """Sequence dst[i] becomes a copy of src[i]'s first ctx tokens: full pages
    shared, the last partial page copied in every layer; ctx[dst] is set."""
    dev, i32 = pool._on_current(), _torch.int32
    n = src.numel()
    rc = load().stv_page_fork(
        ctypes.byref(shape), _layer_array(layers, dev), len(layers), pool._ref, _raw(src, i32, dev, "src"),
        _raw(dst, i32, dev, "dst", n), n, _raw(ctx, i32, dev, "ctx", pool._c.max_seqs),
        _raw(workspace, None, dev, "workspace"), workspace.nbytes, _raw(dev_status, i32, dev, "dev_status"),
        _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_page_fork", rc)


def stv_page_compact(shape, layers, pool: PagePool, page_map, n_live, workspace, dev_status=None, stream=None):
    """Live pages move to the front of every layer's pool, tables and refs
    with them; page_map int32 [n_pages] and n_live int32 [1] are written."""
    dev, i32 = pool._on_current(), _torch.int32
    rc = load().stv_page_compact(
        ctypes.byref(shape), _layer_array(layers, dev), len(layers), pool._ref,
        _raw(page_map, i32, dev, "page_map", pool._c.n_pages), _raw(n_live, i32, dev, "n_live", 1),
        _raw(workspace, None, dev, "workspace"), workspace.nbytes, _raw(dev_status, i32, dev, "dev_status"),
        _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_page_compact", rc)


def stv_page_copy(shape, layers, src, dst, workspace, dev_status=None, stream=None):
    """Page src[i] to page dst[i] in every layer (int32 CUDA tensors); the
    workspace is one for as many pages as the smallest layer's pool has."""
    i32 = _t().int32
    dev = _device_of(workspace, "workspace")
    n = src.numel()
    rc = load().stv_page_copy(
        ctypes.byref(shape), _layer_array(layers, dev), len(layers), min(l.n_pages for l in layers),
        _raw(src, i32, dev, "src"), _raw(dst, i32, dev, "dst", n), n, _raw(workspace, None, dev, "workspace"),
        workspace.nbytes, _raw(dev_status, i32, dev, "dev_status"), _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_page_copy", rc)


# --------------------------------------------------------------------------
# the drafter's side of a round: rows of a ragged batch, a 16-bit paged cache,
# attention over it, acceptance by probabilities
# --------------------------------------------------------------------------

def make_row_shape(hq: int, hkv: int, head_dim: int, dtype) -> stv_shape:
    """The drafter's cache: fp16 or bf16 rows of hkv heads of 64, 128 or 256 channels."""
    torch = _t()
    formats = {torch.float16: STV_KV_ROWS_F16, torch.bfloat16: STV_KV_ROWS_BF16}
    if dtype not in formats:
        raise TypeError(f"the cache's rows must be fp16 or bf16, got {dtype}")
    return stv_shape(int(hq), int(hkv), int(head_dim), 0, PAGE_TOKENS, formats[dtype])


class RowCache:
    """One layer's pool of the drafter's cache: a contiguous CUDA tensor
    [n_pages][hkv][2][256][head_dim] of fp16 or bf16 (K, then V, of each head).
    The page calls take it in the place of a LayerCache."""

    def __init__(self, pool):
        torch = _t()
        if not isinstance(pool, torch.Tensor) or pool.dim() != 5 or pool.shape[2] != 2 or pool.shape[3] != PAGE_TOKENS:
            raise ValueError("the pool must be [n_pages][hkv][2][256][head_dim]")
        if pool.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"the pool must be fp16 or bf16, got {pool.dtype}")
        self.pool = pool
        self.n_pages, self.hkv, _, _, self.head_dim = pool.shape
        self.page_bytes = self.hkv * 4 * PAGE_TOKENS * self.head_dim

    @classmethod
    def empty(cls, n_pages: int, hkv: int, head_dim: int, dtype, device="cuda"):
        return cls(_t().zeros((n_pages, hkv, 2, PAGE_TOKENS, head_dim), dtype=dtype, device=device))

    def c(self) -> stv_layer_cache:
        return stv_layer_cache(_ptr(self.pool, name="pool").value, self.page_bytes, self.n_pages)


def _row_cache(shape, layer, dev):
    """The layer as the calls take it, and its type; the tensor must be what the shape says."""
    pool, fmt = layer.pool, shape.kv_format
    if not isinstance(pool, _torch.Tensor) or pool.get_device() != dev or not pool.is_contiguous():
        raise ValueError(f"the layer's pool must be a contiguous CUDA tensor on cuda:{dev}")
    if layer.hkv != shape.hkv or layer.head_dim != shape.head_dim:
        raise ValueError(f"the shape has {shape.hkv} heads of {shape.head_dim}, the pool {layer.hkv} of {layer.head_dim}")
    dt = pool.dtype
    if fmt != (STV_KV_ROWS_F16 if dt == _torch.float16 else STV_KV_ROWS_BF16 if dt == _torch.bfloat16 else -1):
        raise TypeError(f"the shape's cache format is {fmt}, the pool holds {dt}")
    return struct.pack("@Pqi4x", pool.data_ptr(), layer.page_bytes, layer.n_pages), dt


def make_attn(window: int = 0, sinks: int = 0, causal: bool = True, scale: float = 0.0) -> stv_attn_spec:
    """Which keys a row sees (include/stv.h): window 0: all before it; sinks:
    first tokens that stay visible; causal False: the rows of a block see one
    another; scale 0: head_dim ** -0.5."""
    return stv_attn_spec(int(window), int(sinks), int(bool(causal)), float(scale))


def stv_page_extend(pool: PagePool, seqs, n_new, ctx, row_start, row_seq=None, row_pos=None, slots=None,
                    dev_status=None, stream=None):
    """Pages for n_new[i] more tokens of sequence seqs[i] (None: sequence i),
    and the rows' places: row_start int32 [n + 1]; row_seq, row_pos and slots
    int32 [max_rows], each or None (include/stv.h)."""
    dev, i32 = pool._on_current(), _torch.int32
    n = n_new.numel()
    first = next((t for t in (row_seq, row_pos, slots) if t is not None), None)
    rows = first.numel() if first is not None else 1 << 26
    rc = load().stv_page_extend(
        pool._ref, _raw(seqs, i32, dev, "seqs", n), n, _raw(n_new, i32, dev, "n_new"),
        _raw(ctx, i32, dev, "ctx", pool._c.max_seqs), _raw(row_start, i32, dev, "row_start", n + 1),
        _raw(row_seq, i32, dev, "row_seq", rows), _raw(row_pos, i32, dev, "row_pos", rows),
        _raw(slots, i32, dev, "slots", rows), rows, _raw(dev_status, i32, dev, "dev_status"),
        _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_page_extend", rc)


def stv_kv_write(shape, layer: RowCache, k, v, slots, dev_status=None, stream=None):
    """Rows k, v [n_rows][hkv][head_dim] (any row and head strides) into the
    cache at slots, int32 [n_rows] (-1: left out)."""
    _t()
    dev = _device_of(k, "k")
    lc, dt = _row_cache(shape, layer, dev)
    n, hd = slots.numel(), shape.head_dim
    rc = load().stv_kv_write(
        ctypes.byref(shape), lc, _rows(k, n, hd, dt, dev, "k"), _rows(v, n, hd, dt, dev, "v"),
        _raw(slots, _torch.int32, dev, "slots"), n, _raw(dev_status, _torch.int32, dev, "dev_status"),
        _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_kv_write", rc)


def stv_paged_attn_workspace_bytes(shape, max_new: int) -> int:
    out = ctypes.c_size_t()
    _check("stv_paged_attn_workspace_bytes", load().stv_paged_attn_workspace_bytes(
        ctypes.byref(shape), int(max_new), ctypes.byref(out)))
    return out.value


def stv_paged_attn(shape, spec: stv_attn_spec, layer: RowCache, pool: PagePool, seqs, ctx, row_start, max_new: int, q,
                   o, workspace, dev_status=None, stream=None):
    """Attention of the new rows of n sequences over the drafter's cache.  q, o
    [n_rows][hq][head_dim] (any row and head strides); entry i is sequence
    seqs[i] (None: sequence i) with the rows row_start[i] .. row_start[i + 1] - 1
    (int32 [n + 1]; None: one row each) at positions ctx[s] and on; no entry has
    more than max_new rows (include/stv.h)."""
    _paged_attn("stv_paged_attn", shape, spec, layer, pool, seqs, ctx, row_start, max_new, q, o, workspace, dev_status,
                stream)


def stv_paged_attn_timeout_test(shape, spec: stv_attn_spec, layer: RowCache, pool: PagePool, seqs, ctx, row_start,
                                max_new: int, q, o, workspace, dev_status=None, stream=None):
    """stv_paged_attn with the kernel's copies withheld: every wait runs out
    and the kernel reports STV_DEV_TIMEOUT (failure-path test)."""
    _paged_attn("stv_paged_attn_timeout_test", shape, spec, layer, pool, seqs, ctx, row_start, max_new, q, o, workspace,
                dev_status, stream)


def _paged_attn(fn, shape, spec, layer, pool, seqs, ctx, row_start, max_new, q, o, workspace, dev_status, stream):
    i32 = _t().int32
    dev = pool._on_current()
    lc, dt = _row_cache(shape, layer, dev)
    n_rows, hd = q.shape[0], shape.head_dim
    n = row_start.numel() - 1 if row_start is not None else seqs.numel() if seqs is not None else n_rows
    rc = getattr(load(), fn)(
        ctypes.byref(shape), ctypes.byref(spec), lc, pool._ref, _raw(seqs, i32, dev, "seqs", n), n,
        _raw(ctx, i32, dev, "ctx", pool._c.max_seqs), _raw(row_start, i32, dev, "row_start"), int(max_new),
        _rows(q, n_rows, hd, dt, dev, "q"), _rows(o, n_rows, hd, dt, dev, "o"), n_rows,
        _raw(workspace, None, dev, "workspace"), workspace.nbytes, _raw(dev_status, i32, dev, "dev_status"),
        _raw_stream(stream, dev))
    if rc:
        raise StvError(fn, rc)


def stv_tree_accept_probs(parent, draft_ids, p, q, u, n_commit, path, out_ids, distinct: bool = False,
                          dev_status=None, stream=None):
    """Verification of drafted tokens against the target's probabilities:
    parent, draft_ids int32 [n_seqs][T]; p and q [n_seqs * T][vocab] (fp32,
    fp16 or bf16, rows any distance apart; q None: drafts without a
    distribution); u fp32 [n_seqs][T]; distinct: a node's children were drawn
    without replacement (include/stv.h)."""
    torch = _t()
    dev = _device_of(p, "p")
    if parent.dim() != 2:
        raise ValueError("parent must be [n_seqs][T]")
    n, t = parent.shape
    m = n * t
    if p.dim() != 2 or p.shape[0] != m or (p.shape[1] > 1 and p.stride(1) != 1):
        raise ValueError(f"p must be [{m}][vocab] with adjacent columns")
    vocab, q_at, q_stride = p.shape[1], None, 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.get_device() != dev:
            raise ValueError(f"q must be a CUDA tensor on cuda:{dev}")
        if q.dtype != p.dtype:
            raise TypeError(f"q must be {p.dtype} as p is, got {q.dtype}")
        if tuple(q.shape) != (m, vocab) or (vocab > 1 and q.stride(1) != 1):
            raise ValueError(f"q must be [{m}][{vocab}] with adjacent columns")
        q_at, q_stride = q.data_ptr(), q.stride(0) if m > 1 else vocab
    i32 = torch.int32
    rc = load().stv_tree_accept_probs(
        _raw(parent, i32, dev, "parent"), _raw(draft_ids, i32, dev, "draft_ids", m), p.data_ptr(),
        p.stride(0) if m > 1 else vocab, q_at, q_stride, _dtype_code(p.dtype, "p"), vocab, 1 if distinct else 0,
        _raw(u, torch.float32, dev, "u", m), t, n, _raw(n_commit, i32, dev, "n_commit", n),
        _raw(path, i32, dev, "path", m), _raw(out_ids, i32, dev, "out_ids", m),
        _raw(dev_status, i32, dev, "dev_status"), _raw_stream(stream, dev))
    if rc:
        raise StvError("stv_tree_accept_probs", rc)
