"""Python binding of librq (ResidualQuant KV cache + decode attention on GB300).

Argument marshalling only: every function calls the C entry point of the same
name in librq.so (declared in include/rq.h).  Tensors are passed by device
pointer; streams by handle.  There is no fallback: if the library is missing
this module raises on import.  Build it with
`python decode_attention_rq_gb300/build.py` (nvcc, sm_103a).
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "RQ_OK", "RQ_MODE_SHARED", "RQ_MODE_CHAINED", "RQ_MODE_NORM_RATIO", "RQ_MODE_HADAMARD", "RqError", "rq_config",
    "lib", "LIB_PATH",
    "rq_cache_bytes", "rq_cache_create", "rq_cache_destroy", "rq_append",
    "rq_decode_workspace_bytes", "rq_decode_attention", "rq_bf16_workspace_bytes",
    "rq_decode_attention_bf16", "rq_status_string", "EXPORTED_SYMBOLS",
    "rq_decode_attention_noalloc", "RQ_NOALLOC_WORKSPACE_BYTES", "rq_decode_attention_append",
    "rq_cache_paged_bytes", "rq_cache_create_paged",
    "rq_tree_workspace_bytes", "rq_tree_attention", "RQ_MAX_TREE_NODES",
    "rq_pages_workspace_bytes", "rq_pages_copy", "rq_pages_fork", "rq_pages_reserve", "rq_pages_free",
    "rq_pages_compact",
    "rq_rope", "rq_rope_config", "RQ_ROPE_PLAIN", "RQ_ROPE_LINEAR", "RQ_ROPE_BASE", "RQ_ROPE_PARTS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librq.so")

RQ_OK = 0
RQ_MODE_SHARED = 0
RQ_MODE_CHAINED = 1
RQ_MODE_NORM_RATIO = 2   # flag: norm-ratio coefficient instead of least squares
RQ_MODE_HADAMARD = 4     # flag: R = H_d / sqrt(d) as a fast Walsh-Hadamard transform (d = 128); R_dev may be None
_STATUS_NAMES = {0: "RQ_OK", 1: "RQ_ERR_INVALID_ARG", 2: "RQ_ERR_ALIGNMENT", 3: "RQ_ERR_CAPACITY",
                 4: "RQ_ERR_WORKSPACE", 5: "RQ_ERR_CUDA", 6: "RQ_ERR_UNSUPPORTED", 7: "RQ_ERR_TIMEOUT"}

EXPORTED_SYMBOLS = (
    "rq_cache_bytes", "rq_cache_create", "rq_cache_destroy", "rq_append",
    "rq_decode_workspace_bytes", "rq_decode_attention", "rq_bf16_workspace_bytes",
    "rq_decode_attention_bf16", "rq_status_string", "rq_decode_attention_noalloc",
    "rq_decode_attention_append", "rq_cache_paged_bytes", "rq_cache_create_paged",
    "rq_tree_workspace_bytes", "rq_tree_attention", "rq_pages_workspace_bytes", "rq_pages_copy",
    "rq_pages_fork", "rq_pages_reserve", "rq_pages_free", "rq_pages_compact", "rq_rope",
)

# size of the workspace built into the library for rq_decode_attention_noalloc (rq.h)
RQ_NOALLOC_WORKSPACE_BYTES = 2 * 1024 * 1024
# drafted tokens per row that one rq_tree_attention call may cover (rq.h)
RQ_MAX_TREE_NODES = 256
# frequency scalings of rq_rope (rq.h)
RQ_ROPE_PLAIN, RQ_ROPE_LINEAR, RQ_ROPE_BASE, RQ_ROPE_PARTS = 0, 1, 2, 3


class RqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {_STATUS_NAMES.get(status, status)} ({rq_status_string(status)})")


class rq_config(ctypes.Structure):
    """rq.h's rq_config; num_query_heads (last, default 0) > num_heads selects grouped-query attention."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_layers", "loops_per_group", "num_groups", "num_heads", "head_dim", "group_size",
        "max_batch", "max_seq_len", "mode", "num_query_heads")]


class rq_rope_config(ctypes.Structure):
    """rq.h's rq_rope_config: how rq_rope turns a head."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "head_dim", "rotary_dim", "interleaved", "inverse", "scaling", "original_len")] + [
        (n, ctypes.c_double) for n in ("theta", "factor", "low_turns", "high_turns", "magnitude")]


class _rope_tensor(ctypes.Structure):
    """rq.h's rq_rope_tensor."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int32)] + [
        (n, ctypes.c_int64) for n in ("in_row", "in_head", "in_token", "out_row", "out_head", "out_token")]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python decode_attention_rq_gb300/build.py`")
lib = ctypes.CDLL(LIB_PATH)

_p, _i32, _sz, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
_cfgp = ctypes.POINTER(rq_config)
lib.rq_cache_bytes.argtypes = [_cfgp]
lib.rq_cache_bytes.restype = _sz
lib.rq_cache_create.argtypes = [_cfgp, _p, _sz, _p, ctypes.POINTER(_p)]
lib.rq_cache_create.restype = ctypes.c_int
lib.rq_cache_paged_bytes.argtypes = [_cfgp, _i32]
lib.rq_cache_paged_bytes.restype = _sz
lib.rq_cache_create_paged.argtypes = [_cfgp, _i32, _p, _sz, _p, _i32, _p, ctypes.POINTER(_p)]
lib.rq_cache_create_paged.restype = ctypes.c_int
lib.rq_cache_destroy.argtypes = [_p]
lib.rq_cache_destroy.restype = ctypes.c_int
lib.rq_append.argtypes = [_p, _i32, _i32, _i32, _p, _p, _i32, _p, _p]
lib.rq_append.restype = ctypes.c_int
lib.rq_decode_workspace_bytes.argtypes = [_cfgp, _i32]
lib.rq_decode_workspace_bytes.restype = _sz
lib.rq_decode_attention.argtypes = [_p, _i32, _i32, _i32, _i32, _p, _p, _p, _p, _f, _p, _p, _sz, _p]
lib.rq_decode_attention.restype = ctypes.c_int
lib.rq_decode_attention_noalloc.argtypes = [_p, _i32, _i32, _i32, _i32, _p, _p, _p, _p, _f, _p, _p, _p]
lib.rq_decode_attention_noalloc.restype = ctypes.c_int
lib.rq_decode_attention_append.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _f, _p, _p, _sz, _p]
lib.rq_decode_attention_append.restype = ctypes.c_int
lib.rq_bf16_workspace_bytes.argtypes = [_i32, _i32, _i32]
lib.rq_bf16_workspace_bytes.restype = _sz
lib.rq_decode_attention_bf16.argtypes = [_p, _p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _f, _p, _p, _sz, _p]
lib.rq_decode_attention_bf16.restype = ctypes.c_int
lib.rq_tree_workspace_bytes.argtypes = [_cfgp, _i32, _i32]
lib.rq_tree_workspace_bytes.restype = _sz
lib.rq_tree_attention.argtypes = [_p, _i32, _i32, _i32, _i32, _i32, _p, _p, _p, _p, _p, _p, _f, _p, _p, _sz, _p]
lib.rq_tree_attention.restype = ctypes.c_int
lib.rq_pages_workspace_bytes.argtypes = [_cfgp, _i32]
lib.rq_pages_workspace_bytes.restype = _sz
lib.rq_pages_copy.argtypes = [_p, _i32, _p, _p, _p, _p]
lib.rq_pages_copy.restype = ctypes.c_int
lib.rq_pages_fork.argtypes = [_p, _i32, _p, _p, _p, _p, _p]
lib.rq_pages_fork.restype = ctypes.c_int
lib.rq_pages_reserve.argtypes = [_p, _i32, _p, _i32, _p, _p, _p, _sz, _p]
lib.rq_pages_reserve.restype = ctypes.c_int
lib.rq_pages_free.argtypes = [_p, _i32, _p, _p, _p, _p, _p]
lib.rq_pages_free.restype = ctypes.c_int
lib.rq_pages_compact.argtypes = [_p, _p, _p, _p, _p, _sz, _p]
lib.rq_pages_compact.restype = ctypes.c_int
_ropep = ctypes.POINTER(_rope_tensor)
lib.rq_rope.argtypes = [ctypes.POINTER(rq_rope_config), _i32, _i32, _i32, _ropep, _ropep, _p, _p, _p]
lib.rq_rope.restype = ctypes.c_int
lib.rq_status_string.argtypes = [ctypes.c_int]
lib.rq_status_string.restype = ctypes.c_char_p


def _ptr(x):
    """Device/host address of a tensor (data_ptr) or an int; None -> NULL."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn, st):
    if st != RQ_OK:
        raise RqError(fn, st)


def rq_status_string(status: int) -> str:
    return lib.rq_status_string(status).decode()


def rq_cache_bytes(cfg: rq_config) -> int:
    return lib.rq_cache_bytes(ctypes.byref(cfg))


# What the calls below need of a handle's cache to tell whether a tensor is long enough:
# handle -> (KV heads, query heads, head width, rows, pages; contiguous: 0 pages)
_caches = {}


def _keep(handle, cfg, pages):
    _caches[handle] = (cfg.num_heads, cfg.num_query_heads or cfg.num_heads, cfg.head_dim, cfg.max_batch, pages)
    return handle


def rq_cache_create(cfg: rq_config, dev_buf, nbytes: int, R_dev) -> int:
    """Returns the opaque handle (int)."""
    h = _p()
    _check("rq_cache_create", lib.rq_cache_create(ctypes.byref(cfg), _ptr(dev_buf), nbytes, _ptr(R_dev),
                                                  ctypes.byref(h)))
    return _keep(h.value, cfg, 0)


def rq_cache_paged_bytes(cfg: rq_config, num_pages: int) -> int:
    return lib.rq_cache_paged_bytes(ctypes.byref(cfg), num_pages)


def rq_cache_create_paged(cfg: rq_config, num_pages: int, pool, nbytes: int, block_table, max_tiles_per_row: int,
                          R_dev) -> int:
    """Paged layout: tile t of row b lives in page block_table[b, t] of each
    (layer, group)'s pool.  Returns the opaque handle (int)."""
    h = _p()
    _check("rq_cache_create_paged", lib.rq_cache_create_paged(
        ctypes.byref(cfg), num_pages, _ptr(pool), nbytes, _ptr(block_table), max_tiles_per_row, _ptr(R_dev),
        ctypes.byref(h)))
    return _keep(h.value, cfg, num_pages)


def rq_cache_destroy(handle: int) -> None:
    _caches.pop(handle, None)     # first: once it is destroyed, another thread may be given the same address
    _check("rq_cache_destroy", lib.rq_cache_destroy(handle))


def rq_append(handle, layer, group, batch, kv, seq_lens, n_tokens, status=None, stream=None):
    _check("rq_append", lib.rq_append(handle, layer, group, batch, _ptr(kv), _ptr(seq_lens), n_tokens,
                                      _ptr(status), _stream(stream)))


def rq_decode_workspace_bytes(cfg: rq_config, batch: int) -> int:
    return lib.rq_decode_workspace_bytes(ctypes.byref(cfg), batch)


def rq_decode_attention(handle, layer, group, loop, batch, q, k_cur, v_cur, seq_lens, softmax_scale,
                        out, workspace, workspace_bytes, stream=None):
    _check("rq_decode_attention", lib.rq_decode_attention(
        handle, layer, group, loop, batch, _ptr(q), _ptr(k_cur), _ptr(v_cur), _ptr(seq_lens),
        softmax_scale, _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)))


def rq_decode_attention_append(handle, layer, group, batch, q, kv_cur, seq_lens, softmax_scale, out, workspace,
                               workspace_bytes, stream=None):
    """Anchor-loop attention call that also appends the current token of every
    loop (kv_cur: [P, 2, batch, H, d] bf16) at position seq_lens[b]."""
    _check("rq_decode_attention_append", lib.rq_decode_attention_append(
        handle, layer, group, batch, _ptr(q), _ptr(kv_cur), _ptr(seq_lens), softmax_scale, _ptr(out),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def rq_decode_attention_noalloc(handle, layer, group, loop, batch, q, k_cur, v_cur, seq_lens, softmax_scale,
                                out, status=None, stream=None):
    """rq_decode_attention without a caller workspace, for callers that cannot
    allocate device memory: the scratch lives in a fixed array inside the library
    (RQ_NOALLOC_WORKSPACE_BYTES).  Calls that overlap on the GPU race on it."""
    _check("rq_decode_attention_noalloc", lib.rq_decode_attention_noalloc(
        handle, layer, group, loop, batch, _ptr(q), _ptr(k_cur), _ptr(v_cur), _ptr(seq_lens),
        softmax_scale, _ptr(out), _ptr(status), _stream(stream)))


def rq_bf16_workspace_bytes(batch: int, num_heads: int, head_dim: int) -> int:
    return lib.rq_bf16_workspace_bytes(batch, num_heads, head_dim)


def rq_decode_attention_bf16(k_cache, v_cache, k_cur, v_cur, q, seq_lens, batch, num_heads, head_dim,
                             max_seq, softmax_scale, out, workspace, workspace_bytes, stream=None):
    _check("rq_decode_attention_bf16", lib.rq_decode_attention_bf16(
        _ptr(k_cache), _ptr(v_cache), _ptr(k_cur), _ptr(v_cur), _ptr(q), _ptr(seq_lens), batch,
        num_heads, head_dim, max_seq, softmax_scale, _ptr(out), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def _setup():
    """torch and what the argument checks below compare with, once: a call of a
    few microseconds on the device should not wait for its marshalling."""
    global _torch, _DT, _ROPE_DT
    import torch
    _DT = {"i32": (torch.int32,), "bf16": (torch.bfloat16,), "u64": (torch.int64, torch.uint64), "u8": (torch.uint8,)}
    _ROPE_DT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    _torch = torch


_torch = None


def _device():
    if _torch is None:
        _setup()
    return _torch.cuda.current_device()


def _arg(fn, dev, x, kind, count):
    """Address of x for a C call.  None and ints (device addresses) pass as they
    are; a tensor has to be contiguous, of the kind's dtype, on device dev (the one
    current on this thread) and at least `count` long: a host pointer or a short buffer
    would fault the device."""
    if x is None or isinstance(x, int):
        return x
    if x.dtype not in _DT[kind] or x.get_device() != dev or x.numel() < count or not x.is_contiguous():
        raise RqError(fn, 1)
    return x.data_ptr()


def _pages(handle):
    """Pages of the handle's cache: the length of refs."""
    return _caches.get(handle, (0,) * 5)[4]


def rq_tree_workspace_bytes(cfg: rq_config, batch: int, n_nodes: int) -> int:
    return lib.rq_tree_workspace_bytes(ctypes.byref(cfg), batch, n_nodes)


def rq_tree_attention(handle, layer, group, loop, batch, n_nodes, q, k_new, v_new, mask, node_counts, seq_lens,
                      softmax_scale, out, workspace, workspace_bytes, stream=None):
    """Attention of n_nodes drafted tokens per row (a tree, its visibility in mask)
    over the cached tokens and the draft.  q, out: [batch, Hq, n_nodes, d] bf16;
    k_new, v_new: [batch, H, n_nodes, d] bf16; mask: [batch, n_nodes,
    ceil(n_nodes / 64)] int64 or uint64 bits, or None (a single sequence);
    node_counts: [batch] int32 or None."""
    fn, dev = "rq_tree_attention", _device()
    cache = _caches.get(handle)
    if cache is None:     # a handle made without this binding: one head of the smaller width, out as q, v_new as k_new
        nq, nk = (max(batch * n_nodes * 96, 0 if x is None or isinstance(x, int) else x.numel()) for x in (q, k_new))
    elif batch > cache[3] or n_nodes > RQ_MAX_TREE_NODES:     # the library refuses these before it reads anything
        nq = nk = 0
    else:
        nodes = batch * n_nodes * cache[2]
        nk, nq = nodes * cache[0], nodes * cache[1]
    _check(fn, lib.rq_tree_attention(
        handle, layer, group, loop, batch, n_nodes, _arg(fn, dev, q, "bf16", nq),
        _arg(fn, dev, k_new, "bf16", nk), _arg(fn, dev, v_new, "bf16", nk),
        _arg(fn, dev, mask, "u64", batch * n_nodes * -(-n_nodes // 64)),
        _arg(fn, dev, node_counts, "i32", batch), _arg(fn, dev, seq_lens, "i32", batch), softmax_scale,
        _arg(fn, dev, out, "bf16", nq), _arg(fn, dev, workspace, "u8", workspace_bytes), workspace_bytes,
        _stream(stream)))


def rq_pages_workspace_bytes(cfg: rq_config, num_pages: int) -> int:
    return lib.rq_pages_workspace_bytes(ctypes.byref(cfg), num_pages)


def rq_pages_copy(handle, n, src, dst, status=None, stream=None):
    """Copy page src[i] to page dst[i] of a paged cache, every layer and group."""
    fn, dev = "rq_pages_copy", _device()
    _check(fn, lib.rq_pages_copy(
        handle, n, _arg(fn, dev, src, "i32", n), _arg(fn, dev, dst, "i32", n), _arg(fn, dev, status, "i32", 4),
        _stream(stream)))


def rq_pages_fork(handle, n, src_rows, dst_rows, refs, status=None, stream=None):
    """Row dst_rows[i] shares the pages of row src_rows[i] and gives up its own."""
    fn, dev = "rq_pages_fork", _device()
    _check(fn, lib.rq_pages_fork(
        handle, n, _arg(fn, dev, src_rows, "i32", n), _arg(fn, dev, dst_rows, "i32", n),
        _arg(fn, dev, refs, "i32", _pages(handle)), _arg(fn, dev, status, "i32", 4), _stream(stream)))


def rq_pages_reserve(handle, batch, seq_lens, n_tokens, refs, status, workspace, workspace_bytes, stream=None):
    """Give rows 0 .. batch-1 pages of their own for their next n_tokens positions
    (copy on write where a page is shared)."""
    fn, dev = "rq_pages_reserve", _device()
    _check(fn, lib.rq_pages_reserve(
        handle, batch, _arg(fn, dev, seq_lens, "i32", batch), n_tokens,
        _arg(fn, dev, refs, "i32", _pages(handle)),
        _arg(fn, dev, status, "i32", 4), _arg(fn, dev, workspace, "u8", workspace_bytes), workspace_bytes,
        _stream(stream)))


def rq_pages_free(handle, n, rows, keep, refs, status=None, stream=None):
    """Give up the pages of rows[i] behind its first keep[i] tokens (keep None: all)."""
    fn, dev = "rq_pages_free", _device()
    _check(fn, lib.rq_pages_free(
        handle, n, _arg(fn, dev, rows, "i32", n), _arg(fn, dev, keep, "i32", n),
        _arg(fn, dev, refs, "i32", _pages(handle)),
        _arg(fn, dev, status, "i32", 4), _stream(stream)))


def rq_pages_compact(handle, refs, used, status, workspace, workspace_bytes, stream=None):
    """Move the used pages to the front of the pool; used (int32 on the device)
    receives their number."""
    fn, dev = "rq_pages_compact", _device()
    _check(fn, lib.rq_pages_compact(
        handle, _arg(fn, dev, refs, "i32", _pages(handle)), _arg(fn, dev, used, "i32", 1),
        _arg(fn, dev, status, "i32", 4), _arg(fn, dev, workspace, "u8", workspace_bytes), workspace_bytes,
        _stream(stream)))


def rq_rope(cfg: rq_rope_config, q, k, start, offsets=None, q_out=None, k_out=None, stream=None):
    """Rotate q and k ([batch, heads, n, d] tensors of any strides with contiguous
    channels; either may be None) by positions start[b] + offsets[b, t] (offsets
    None: + t).  q_out, k_out None: in place."""
    fn, dev = "rq_rope", _device()
    first = q if q is not None else k
    if first is None or first.dim() != 4 or first.dtype not in _ROPE_DT:
        raise RqError(fn, 1)
    dtype = first.dtype
    batch, _, n, _ = first.shape

    def pack(x, y):
        if x is None:
            return None
        shape, xs = x.shape, x.stride()
        if (len(shape) != 4 or x.dtype is not dtype or shape[0] != batch or shape[2] != n or shape[3] != cfg.head_dim
                or xs[3] != 1 or x.get_device() != dev):
            raise RqError(fn, 1)
        if y is None or y is x:
            y, ys = x, xs
        else:
            ys = y.stride()
            if y.dtype is not dtype or y.shape != shape or ys[3] != 1 or y.get_device() != dev:
                raise RqError(fn, 1)
        return _rope_tensor(x.data_ptr(), y.data_ptr(), shape[1], xs[0], xs[1], xs[2], ys[0], ys[1], ys[2])

    tq, tk = pack(q, q_out), pack(k, k_out)
    _check(fn, lib.rq_rope(ctypes.byref(cfg), _ROPE_DT[dtype], batch, n, None if tq is None else ctypes.byref(tq),
                           None if tk is None else ctypes.byref(tk), _arg(fn, dev, start, "i32", batch),
                           _arg(fn, dev, offsets, "i32", batch * n), _stream(stream)))
