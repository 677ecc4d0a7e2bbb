"""Token log-probabilities and surprisal (sekv_token_logprobs, sekv_surprisal):
argument marshalling only."""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from .sekv import DTYPES, Workspace, _check, _ptr, _stream, check_tensor, lib


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor                  # f32, tokens' shape
    lse: Optional[torch.Tensor]            # f32
    entropy: Optional[torch.Tensor]        # f32
    top_ids: Optional[torch.Tensor]        # int32 [...][n_top]
    top_logprobs: Optional[torch.Tensor]   # f32 [...][n_top]


def _rows(logits, tokens):
    """(batch, rows of a sequence, strides of logits and tokens) of [T][V] or [B][T][V] logits."""
    if logits.dim() not in (2, 3) or logits.stride(-1) != 1:
        raise ValueError(f"logits: expected [T][V] or [B][T][V] with consecutive entries, got "
                         f"{tuple(logits.shape)}")
    check_tensor(logits, "logits", tuple(DTYPES), logits.device)
    check_tensor(tokens, "tokens", (torch.int32, torch.int64), logits.device)
    if tokens.shape != logits.shape[:-1] or (tokens.shape[-1] > 1 and tokens.stride(-1) != 1):
        raise ValueError(f"tokens: expected {tuple(logits.shape[:-1])} with consecutive entries, "
                         f"got {tuple(tokens.shape)}")
    if logits.dim() == 2:
        return 1, logits.shape[0], 0, logits.stride(0), 0
    return (logits.shape[0], logits.shape[1], logits.stride(0), logits.stride(1),
            tokens.stride(0))


def _check_ws(ws, dev):
    if ws.buf.device != dev:
        raise ValueError(f"workspace: on {ws.buf.device}, tensors on {dev}")


def token_logprobs(logits, tokens, ws: Workspace, n_top: int = 0, scale: float = 1.0,
                   entropy: bool = True, stream=None) -> TokenLogprobs:
    """Log-probabilities of `tokens` ([T] or [B][T], -1: none) under `logits`
    ([T][V] or [B][T][V]; bf16, f16 or f32) times `scale` (1 / temperature), with
    log-sum-exp and entropy (entropy=False: neither) and the n_top (at most 32)
    likeliest tokens.  `ws` is any workspace: bad token ids go to its status."""
    B, T, sb, st, tb = _rows(logits, tokens)
    dev = logits.device
    _check_ws(ws, dev)
    shape = tokens.shape
    lp = torch.empty(shape, dtype=torch.float32, device=dev)
    lse = ent = ids = tlp = None
    if entropy:
        lse, ent = torch.empty((2, *shape), dtype=torch.float32, device=dev).unbind(0)
    if n_top > 0:
        ids = torch.empty((*shape, n_top), dtype=torch.int32, device=dev)
        tlp = torch.empty((*shape, n_top), dtype=torch.float32, device=dev)
    if lp.numel():
        _check("sekv_token_logprobs",
               lib().sekv_token_logprobs(logits.data_ptr(), DTYPES[logits.dtype], B, T,
                                         logits.shape[-1], sb, st, tokens.data_ptr(),
                                         tokens.dtype == torch.int64, tb, scale, n_top,
                                         lp.data_ptr(), _ptr(lse), _ptr(ent), _ptr(ids),
                                         _ptr(tlp), ws.ptr(), ws.nbytes, _stream(stream)))
    return TokenLogprobs(lp, lse, ent, ids, tlp)


def surprisal(logits, tokens, ws: Workspace, out=None, stream=None):
    """H [B][T] f32 of the sequences `tokens` [B][T] under `logits` [B][T][V]: -log p of
    each token given those before it, 0 for the first; what build_spans takes."""
    if logits.dim() != 3:
        raise ValueError(f"logits: expected [B][T][V], got {tuple(logits.shape)}")
    B, T, sb, st, tb = _rows(logits, tokens)
    dev = logits.device
    _check_ws(ws, dev)
    if out is None:
        out = torch.empty(B, T, dtype=torch.float32, device=dev)
    else:
        check_tensor(out, "out", (torch.float32,), dev)
        if out.shape != (B, T) or not out.is_contiguous():
            raise ValueError(f"out: expected contiguous [{B}][{T}], got {tuple(out.shape)}")
    if out.numel():
        _check("sekv_surprisal",
               lib().sekv_surprisal(logits.data_ptr(), DTYPES[logits.dtype], B, T,
                                    logits.shape[-1], sb, st, tokens.data_ptr(),
                                    tokens.dtype == torch.int64, tb, out.data_ptr(), ws.ptr(),
                                    ws.nbytes, _stream(stream)))
    return out
