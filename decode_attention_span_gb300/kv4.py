"""The 4-bit cache (sekv_kv4_append, sekv_kv4_read, sekv_kv4_attention):
argument marshalling only."""

from __future__ import annotations

import ctypes

import torch

from .sekv import DTYPES, Config, Workspace, _check, _ptr, _stream, check_tensor, lib

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
        dev = pages.device
        check_tensor(pages, "pages", (torch.uint8,), dev)
        check_tensor(page_table, "page_table", (torch.int32,), dev)
        if (pages.dim() != 3 or pages.shape[1:] != (cfg.n_kv_heads, PAGE_BYTES) or
                not pages.is_contiguous()):
            raise ValueError(f"pages: expected contiguous [n][{cfg.n_kv_heads}][{PAGE_BYTES}], got "
                             f"{tuple(pages.shape)}")
        if (page_table.dim() != 2 or page_table.shape[0] != cfg.batch or
                not page_table.is_contiguous()):
            raise ValueError(f"page_table: expected contiguous [{cfg.batch}][max_pages], got "
                             f"{tuple(page_table.shape)}")
        self.pages, self.page_table, self.device = pages, page_table, dev
        self.batch, self.n_kv_heads = cfg.batch, cfg.n_kv_heads
        self._c = SekvKv4Cache(pages.data_ptr(), page_table.data_ptr(), pages.shape[0],
                               page_table.shape[1])


def _common(cfg, cache, ws):
    if (cfg.batch, cfg.n_kv_heads) != (cache.batch, cache.n_kv_heads):
        raise ValueError("cache: made for another batch or number of KV heads")
    if ws.buf.device != cache.device:
        raise ValueError(f"workspace: on {ws.buf.device}, cache on {cache.device}")


def _per_seq(t, name, cfg, dev):
    check_tensor(t, name, (torch.int32,), dev)
    if t.shape != (cfg.batch,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous [{cfg.batch}], got {tuple(t.shape)}")
    return t.data_ptr()


_Stride = ctypes.c_int64 * 3


def kv4_append(cfg: Config, cache: Kv4Cache, k, v, first, ws: Workspace, n_valid=None,
               stream=None):
    """Stores k and v [B][T][Hkv][128] (bf16 or f16; any strides that are multiples of
    8 with the last one 1) at token positions first[b] .. first[b] + T - 1 of each
    sequence; with n_valid [B], only its first n_valid[b] rows."""
    _common(cfg, cache, ws)
    dev = cache.device
    check_tensor(k, "k", _HALF, dev)
    check_tensor(v, "v", (k.dtype,), dev)
    for name, x in (("k", k), ("v", v)):
        if (x.dim() != 4 or x.shape != (cfg.batch, k.shape[1], cfg.n_kv_heads, 128) or
                x.stride(3) != 1):
            raise ValueError(f"{name}: expected [{cfg.batch}][T][{cfg.n_kv_heads}][128], got "
                             f"{tuple(x.shape)}")
    f = _per_seq(first, "first", cfg, dev)
    n = None if n_valid is None else _per_seq(n_valid, "n_valid", cfg, dev)
    c = cfg.c()
    _check("sekv_kv4_append",
           lib().sekv_kv4_append(ctypes.byref(c), ctypes.byref(cache._c), DTYPES[k.dtype],
                                 k.data_ptr(), _Stride(*k.stride()[:3]), v.data_ptr(),
                                 _Stride(*v.stride()[:3]), k.shape[1], f, n, ws.ptr(), ws.nbytes,
                                 _stream(stream)))


def kv4_read(cfg: Config, cache: Kv4Cache, first, n_tokens: int, ws: Workspace,
             dtype=torch.bfloat16, n_valid=None, out=None, stream=None):
    """K and V [B][Hkv][n_tokens][128] that the tokens first[b] .. first[b] + n_tokens - 1
    stand for, rounded to dtype (bf16, f16 or f32).  With n_valid [B], rows from
    n_valid[b] on stay as they were (zero in outputs made here)."""
    _common(cfg, cache, ws)
    dev = cache.device
    shape = (cfg.batch, cfg.n_kv_heads, n_tokens, 128)
    if out is None:
        k, v = torch.zeros((2, *shape), dtype=dtype, device=dev).unbind(0)
    else:
        k, v = out
        check_tensor(k, "out[0]", tuple(DTYPES), dev)
        check_tensor(v, "out[1]", (k.dtype,), dev)
        if k.shape != shape or v.shape != shape or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError(f"out: expected contiguous {shape}")
    f = _per_seq(first, "first", cfg, dev)
    n = None if n_valid is None else _per_seq(n_valid, "n_valid", cfg, dev)
    c = cfg.c()
    if n_tokens > 0:
        _check("sekv_kv4_read",
               lib().sekv_kv4_read(ctypes.byref(c), ctypes.byref(cache._c), DTYPES[k.dtype],
                                   k.data_ptr(), v.data_ptr(), n_tokens, f, n, ws.ptr(),
                                   ws.nbytes, _stream(stream)))
    return k, v


def kv4_attention(cfg: Config, cache: Kv4Cache, q, seq_len, scale: float, ws: Workspace,
                  out=None, lse=None, stream=None):
    """Attention of q [B][n_q][Hq][128] (bf16 or f16) over the first seq_len[b] cached
    tokens of each sequence, the query tokens being its last n_q; returns out
    [B][n_q][Hq][128] f32 and lse [B][n_q][Hq] f32."""
    _common(cfg, cache, ws)
    dev = cache.device
    check_tensor(q, "q", _HALF, dev)
    if q.dim() != 4 or q.shape[0] != cfg.batch or q.shape[2:] != (cfg.n_q_heads, 128) or \
            not q.is_contiguous():
        raise ValueError(f"q: expected contiguous [{cfg.batch}][n_q][{cfg.n_q_heads}][128], got "
                         f"{tuple(q.shape)}")
    n_q = q.shape[1]
    for name, t, shape in (("out", out, q.shape), ("lse", lse, q.shape[:3])):
        if t is not None:
            check_tensor(t, name, (torch.float32,), dev)
            if t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous {tuple(shape)}")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev)
    s = _per_seq(seq_len, "seq_len", cfg, dev)
    c = cfg.c()
    _check("sekv_kv4_attention",
           lib().sekv_kv4_attention(ctypes.byref(c), ctypes.byref(cache._c), DTYPES[q.dtype],
                                    q.data_ptr(), n_q, s, scale, out.data_ptr(), lse.data_ptr(),
                                    ws.ptr(), ws.nbytes, _stream(stream)))
    return out, lse
