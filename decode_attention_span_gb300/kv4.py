"""The 4-bit cache (sekv_kv4_append, sekv_kv4_read, sekv_kv4_attention):
argument marshalling only."""

from __future__ import annotations

import ctypes

import torch

from .sekv import (DTYPES, SEKV_CALL_KV4, Config, Workspace, _check, check_tensor, current_index, lib,
                   made_on, raw_stream)

PAGE_TOKENS = 64
PAGE_BYTES = 9216
_HALF = (torch.bfloat16, torch.float16)


class SekvKv4Cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


def alloc_kv4_pages(cfg: Config, n_pages: int, device=None) -> torch.Tensor:
    """A pool of n_pages pages of 64 tokens (uninitialised: pages need none)."""
    return torch.empty(n_pages, cfg.n_kv_heads, PAGE_BYTES, dtype=torch.uint8,
                       device=device or "cuda")


class Kv4Cache:
    """One layer's 4-bit cache: a page pool [n_pages][Hkv][9216] uint8 and the page
    table int32 [B][max_pages] of its sequences (layout in include/sekv.h).  The
    tensors are the caller's; the table may be rewritten between calls."""

    def __init__(self, cfg: Config, pages: torch.Tensor, page_table: torch.Tensor):
        index = current_index(pages, "pages")
        check_tensor(pages, "pages", (torch.uint8,), index)
        check_tensor(page_table, "page_table", (torch.int32,), index)
        if (pages.dim() != 3 or pages.shape[1:] != (cfg.n_kv_heads, PAGE_BYTES) or
                not pages.is_contiguous()):
            raise ValueError(f"pages: expected contiguous [n][{cfg.n_kv_heads}][{PAGE_BYTES}], got "
                             f"{tuple(pages.shape)}")
        if (page_table.dim() != 2 or page_table.shape[0] != cfg.batch or
                not page_table.is_contiguous()):
            raise ValueError(f"page_table: expected contiguous [{cfg.batch}][max_pages], got "
                             f"{tuple(page_table.shape)}")
        self.pages, self.page_table, self.device = pages, page_table, pages.device
        self.batch, self.n_kv_heads = cfg.batch, cfg.n_kv_heads
        self._struct = SekvKv4Cache(pages.data_ptr(), page_table.data_ptr(), pages.shape[0],
                                    page_table.shape[1])
        self._c = ctypes.byref(self._struct)


def _common(cfg, cache, ws) -> int:
    if cfg.batch != cache.batch or cfg.n_kv_heads != cache.n_kv_heads:
        raise ValueError("cache: made for another batch or number of KV heads")
    index = current_index(cache.pages, "pages")
    if ws.which != SEKV_CALL_KV4:
        raise ValueError("workspace: made for another call, expected which=SEKV_CALL_KV4")
    if ws.buf.get_device() != index:
        raise ValueError(f"workspace: on {ws.buf.device}, cache on {cache.device}")
    return index


_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _per_seq(t, name, cfg, index):
    check_tensor(t, name, _I32, index)
    s = t.shape
    if len(s) != 1 or s[0] != cfg.batch or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous [{cfg.batch}], got {tuple(t.shape)}")
    return t.data_ptr()


_Stride = ctypes.c_int64 * 3


def _rows(x, name, dtypes, cfg, n, index):
    check_tensor(x, name, dtypes, index)
    s = x.stride()
    if x.shape != (cfg.batch, n, cfg.n_kv_heads, 128) or s[3] != 1:
        raise ValueError(f"{name}: expected [{cfg.batch}][T][{cfg.n_kv_heads}][128] with "
                         f"consecutive elements in a head, got {tuple(x.shape)}")
    return _Stride(s[0], s[1], s[2])


def kv4_append(cfg: Config, cache: Kv4Cache, k, v, first, ws: Workspace, n_valid=None,
               stream=None):
    """Stores k and v [B][T][Hkv][128] (bf16 or f16; any strides that are multiples of
    8 with the last one 1) at token positions first[b] .. first[b] + T - 1 of each
    sequence; with n_valid [B], only its first n_valid[b] rows."""
    index = _common(cfg, cache, ws)
    T = k.shape[1] if k.dim() == 4 else 0
    ks = _rows(k, "k", _HALF, cfg, T, index)
    vs = _rows(v, "v", (k.dtype,), cfg, T, index)
    f = _per_seq(first, "first", cfg, index)
    n = None if n_valid is None else _per_seq(n_valid, "n_valid", cfg, index)
    st = lib().sekv_kv4_append(ctypes.byref(cfg.c()), cache._c, DTYPES[k.dtype], k.data_ptr(), ks,
                               v.data_ptr(), vs, T, f, n, ws.buf.data_ptr(), ws.nbytes,
                               raw_stream(stream, index))
    if st != 0:
        _check("sekv_kv4_append", st)


def kv4_read(cfg: Config, cache: Kv4Cache, first, n_tokens: int, ws: Workspace,
             dtype=torch.bfloat16, n_valid=None, out=None, stream=None):
    """K and V [B][Hkv][n_tokens][128] that the tokens first[b] .. first[b] + n_tokens - 1
    stand for, rounded to dtype (bf16, f16 or f32).  With n_valid [B], rows from
    n_valid[b] on stay as they were (zero in outputs made here); tokens that the workspace's
    status flags are not written."""
    index = _common(cfg, cache, ws)
    dev = cache.device
    shape = (cfg.batch, cfg.n_kv_heads, n_tokens, 128)
    n = None
    if n_valid is not None:
        n = _per_seq(n_valid, "n_valid", cfg, index)
    if out is None:
        if dtype not in DTYPES:
            raise TypeError(f"dtype: expected one of {list(DTYPES)}, got {dtype}")
        make = torch.empty if n is None else torch.zeros
        with made_on(stream, index):
            k, v = make(shape, dtype=dtype, device=dev), make(shape, dtype=dtype, device=dev)
    else:
        k, v = out
        check_tensor(k, "out[0]", DTYPES, index)
        check_tensor(v, "out[1]", (k.dtype,), index)
        if k.shape != shape or v.shape != shape or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError(f"out: expected contiguous {shape}")
    f = _per_seq(first, "first", cfg, index)
    st = lib().sekv_kv4_read(ctypes.byref(cfg.c()), cache._c, DTYPES[k.dtype], k.data_ptr(),
                             v.data_ptr(), n_tokens, f, n, ws.buf.data_ptr(), ws.nbytes,
                             raw_stream(stream, index))
    if st != 0:
        _check("sekv_kv4_read", st)
    return k, v


def _queries(cfg, cache, q, out, lse, index, stream):
    """(out, lse) of queries [B][n_q][Hq][128], made here where not given."""
    check_tensor(q, "q", _HALF, index)
    shape = q.shape
    if len(shape) != 4 or shape[0] != cfg.batch or shape[2] != cfg.n_q_heads or \
            shape[3] != 128 or not q.is_contiguous():
        raise ValueError(f"q: expected contiguous [{cfg.batch}][n_q][{cfg.n_q_heads}][128], got "
                         f"{tuple(shape)}")
    if out is None:
        with made_on(stream, index):
            out = torch.empty(shape, dtype=torch.float32, device=cache.device)
    else:
        check_tensor(out, "out", _F32, index)
        if out.shape != shape or not out.is_contiguous():
            raise ValueError(f"out: expected contiguous {tuple(shape)}")
    if lse is None:
        with made_on(stream, index):
            lse = torch.empty(shape[:3], dtype=torch.float32, device=cache.device)
    else:
        check_tensor(lse, "lse", _F32, index)
        if lse.shape != shape[:3] or not lse.is_contiguous():
            raise ValueError(f"lse: expected contiguous {tuple(shape[:3])}")
    return out, lse


def kv4_attention(cfg: Config, cache: Kv4Cache, q, seq_len, scale: float, ws: Workspace,
                  out=None, lse=None, stream=None):
    """Attention of q [B][n_q][Hq][128] (bf16 or f16) over the first seq_len[b] cached
    tokens of each sequence, the query tokens being its last n_q; returns out
    [B][n_q][Hq][128] f32 and lse [B][n_q][Hq] f32."""
    index = _common(cfg, cache, ws)
    out, lse = _queries(cfg, cache, q, out, lse, index, stream)
    s = _per_seq(seq_len, "seq_len", cfg, index)
    st = lib().sekv_kv4_attention(ctypes.byref(cfg.c()), cache._c, DTYPES[q.dtype], q.data_ptr(),
                                  q.shape[1], s, scale, out.data_ptr(), lse.data_ptr(),
                                  ws.buf.data_ptr(), ws.nbytes, raw_stream(stream, index))
    if st != 0:
        _check("sekv_kv4_attention", st)
    return out, lse


_I64 = (torch.int64,)


def kv4_tree_attention(cfg: Config, cache: Kv4Cache, q, first, tree, scale: float, ws: Workspace,
                       out=None, lse=None, stream=None):
    """Attention of a tree of drafted tokens: q [B][n_q][Hq][128] (bf16 or f16), stored at positions
    first[b] .. first[b] + n_q - 1, over the first[b] tokens before them and, of the drafted ones, over
    those of the bits of `tree` (int64 [B][n_q], or [n_q] for all sequences: bit j of entry i lets
    token i see token j).  Returns out and lse as kv4_attention does."""
    index = _common(cfg, cache, ws)
    out, lse = _queries(cfg, cache, q, out, lse, index, stream)
    n = q.shape[1]
    check_tensor(tree, "tree", _I64, index)
    if tree.shape not in ((cfg.batch, n), (n,)) or not tree.is_contiguous():
        raise ValueError(f"tree: expected contiguous [{cfg.batch}][{n}] or [{n}], got "
                         f"{tuple(tree.shape)}")
    f = _per_seq(first, "first", cfg, index)
    st = lib().sekv_kv4_tree_attention(ctypes.byref(cfg.c()), cache._c, DTYPES[q.dtype],
                                       q.data_ptr(), n, f, tree.data_ptr(),
                                       n if tree.dim() == 2 else 0, scale, out.data_ptr(),
                                       lse.data_ptr(), ws.buf.data_ptr(), ws.nbytes,
                                       raw_stream(stream, index))
    if st != 0:
        _check("sekv_kv4_tree_attention", st)
    return out, lse


def kv4_keep(cfg: Config, cache: Kv4Cache, first, keep, n_keep, ws: Workspace, stream=None):
    """Keeps a branch of the drafted tokens: token first[b] + keep[b][i] moves to first[b] + i, for
    i < n_keep[b] (None: all); keep int32 [B][n] (n at most 64), ascending."""
    index = _common(cfg, cache, ws)
    check_tensor(keep, "keep", _I32, index)
    if keep.dim() != 2 or keep.shape[0] != cfg.batch or not keep.is_contiguous():
        raise ValueError(f"keep: expected contiguous [{cfg.batch}][n], got {tuple(keep.shape)}")
    f = _per_seq(first, "first", cfg, index)
    n = None if n_keep is None else _per_seq(n_keep, "n_keep", cfg, index)
    st = lib().sekv_kv4_keep(ctypes.byref(cfg.c()), cache._c, f, keep.data_ptr(), keep.shape[1], n,
                             ws.buf.data_ptr(), ws.nbytes, raw_stream(stream, index))
    if st != 0:
        _check("sekv_kv4_keep", st)
