"""Token log-probabilities and surprisal (sekv_token_logprobs, sekv_surprisal):
argument marshalling only."""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from .sekv import DTYPES, Workspace, _check, check_tensor, current_index, lib, made_on, raw_stream


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor                  # f32, tokens' shape
    lse: Optional[torch.Tensor]            # f32
    entropy: Optional[torch.Tensor]        # f32
    top_ids: Optional[torch.Tensor]        # int32 [...][n_top]
    top_logprobs: Optional[torch.Tensor]   # f32 [...][n_top]


_IDS = (torch.int32, torch.int64)


def _rows(logits, tokens, ws):
    """(device index, type, batch, rows of a sequence, vocabulary, strides of logits, stride of
    tokens) of [T][V] or [B][T][V] logits."""
    dtype = DTYPES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits: expected one of {list(DTYPES)}, got {logits.dtype}")
    index = current_index(logits, "logits")
    s, ls = logits.shape, logits.stride()
    n = len(s)
    if n not in (2, 3) or ls[-1] != 1:
        raise ValueError(f"logits: expected [T][V] or [B][T][V] with consecutive entries, got "
                         f"{tuple(s)}")
    check_tensor(tokens, "tokens", _IDS, index)
    ts = tokens.stride()
    if tokens.shape != s[:-1] or (s[-2] > 1 and ts[-1] != 1):
        raise ValueError(f"tokens: expected {tuple(s[:-1])} with consecutive entries, got "
                         f"{tuple(tokens.shape)}")
    if ws.buf.get_device() != index:
        raise ValueError(f"workspace: on {ws.buf.device}, tensors on {logits.device}")
    if n == 2:
        return index, dtype, 1, s[0], s[1], 0, ls[0], 0
    return index, dtype, s[0], s[1], s[2], ls[0], ls[1], ts[0]


def token_logprobs(logits, tokens, ws: Workspace, n_top: int = 0, scale: float = 1.0,
                   entropy: bool = True, stream=None) -> TokenLogprobs:
    """Log-probabilities of `tokens` ([T] or [B][T], -1: none) under `logits`
    ([T][V] or [B][T][V]; bf16, f16 or f32) times `scale` (1 / temperature), with
    log-sum-exp and entropy (entropy=False: neither) and the n_top (at most 32)
    likeliest tokens.  `ws` is any workspace: bad token ids go to its status."""
    index, dtype, B, T, V, sb, st, tb = _rows(logits, tokens, ws)
    shape = tokens.shape
    empty, f32, dev = torch.empty, torch.float32, logits.device
    lse = ent = ids = tlp = None
    p_lse = p_ent = p_ids = p_tlp = None
    with made_on(stream, index):
        lp = empty(shape, dtype=f32, device=dev)
        if entropy:
            lse, ent = empty(shape, dtype=f32, device=dev), empty(shape, dtype=f32, device=dev)
            p_lse, p_ent = lse.data_ptr(), ent.data_ptr()
        if n_top > 0:
            ids = empty((*shape, n_top), dtype=torch.int32, device=dev)
            tlp = empty((*shape, n_top), dtype=f32, device=dev)
            p_ids, p_tlp = ids.data_ptr(), tlp.data_ptr()
    if B * T > 0:
        err = lib().sekv_token_logprobs(logits.data_ptr(), dtype, B, T, V, sb, st,
                                        tokens.data_ptr(), tokens.dtype == torch.int64, tb, scale,
                                        n_top, lp.data_ptr(), p_lse, p_ent, p_ids, p_tlp,
                                        ws.buf.data_ptr(), ws.nbytes, raw_stream(stream, index))
        if err != 0:
            _check("sekv_token_logprobs", err)
    return TokenLogprobs(lp, lse, ent, ids, tlp)


def surprisal(logits, tokens, ws: Workspace, out=None, stream=None):
    """H [B][T] f32 of the sequences `tokens` [B][T] under `logits` [B][T][V]: -log p of
    each token given those before it, 0 for the first; what build_spans takes."""
    if logits.dim() != 3:
        raise ValueError(f"logits: expected [B][T][V], got {tuple(logits.shape)}")
    index, dtype, B, T, V, sb, st, tb = _rows(logits, tokens, ws)
    if out is None:
        with made_on(stream, index):
            out = torch.empty(B, T, dtype=torch.float32, device=logits.device)
    else:
        check_tensor(out, "out", (torch.float32,), index)
        if out.shape != (B, T) or not out.is_contiguous():
            raise ValueError(f"out: expected contiguous [{B}][{T}], got {tuple(out.shape)}")
    if B * T > 0:
        err = lib().sekv_surprisal(logits.data_ptr(), dtype, B, T, V, sb, st, tokens.data_ptr(),
                                   tokens.dtype == torch.int64, tb, out.data_ptr(),
                                   ws.buf.data_ptr(), ws.nbytes, raw_stream(stream, index))
        if err != 0:
            _check("sekv_surprisal", err)
    return out
