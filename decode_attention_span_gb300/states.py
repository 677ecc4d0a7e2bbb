"""Log-probabilities from last states (sekv_states_logprobs, sekv_states_surprisal and the
gradient): argument marshalling only."""

from __future__ import annotations

from typing import NamedTuple

import torch

from .sekv import (DTYPES, SekvError, Workspace, _check, _ptr, _stream, check_tensor,
                   current_index, lib, made_on, raw_stream)

_HALF = (torch.bfloat16, torch.float16)
_IDS = (torch.int32, torch.int64)
_F32 = (torch.float32,)


class StatesWorkspace(Workspace):
    """Scratch of the states_* calls: for up to `rows` rows against up to `vocab` tokens of
    states of up to `dim` elements; `backward` for states_logprobs_backward too."""

    def __init__(self, rows: int, vocab: int, dim: int, backward: bool = False, device=None):
        n = int(lib().sekv_states_workspace_size(rows, vocab, dim, int(backward)))
        if n == 0:
            raise SekvError("sekv_states_workspace_size", -1)
        self.nbytes, self.which = n, "states"
        self.buf = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
        _check("sekv_workspace_init", lib().sekv_workspace_init(_ptr(self.buf), n, _stream()))


class StatesLogprobs(NamedTuple):
    logprob: torch.Tensor  # f32, tokens' shape
    lse: torch.Tensor      # f32


def _rows(states, weight, tokens, ws):
    """(device index, type, rows, dimensions, stride of a state, vocabulary, stride of a weight)."""
    index = current_index(states, "states")
    check_tensor(states, "states", _HALF, index)
    check_tensor(weight, "weight", (states.dtype,), index)
    s, x = states.shape, states.stride()
    if len(s) not in (2, 3) or (x[-1] != 1 and s[-1] > 1):
        raise ValueError(f"states: expected [T][D] or [B][T][D] with consecutive elements, got "
                         f"{tuple(s)}")
    stride = x[-2]
    if len(s) == 3:
        if s[1] == 1:
            stride = x[0]
        elif s[0] > 1 and x[0] != s[1] * x[1]:
            raise ValueError("states: rows have to be evenly spaced over the sequences")
    w = weight.stride()
    if weight.dim() != 2 or weight.shape[1] != s[-1] or (w[1] != 1 and s[-1] > 1):
        raise ValueError(f"weight: expected [V][{s[-1]}] with consecutive elements, got "
                         f"{tuple(weight.shape)}")
    check_tensor(tokens, "tokens", _IDS, index)
    if tokens.shape != s[:-1] or not tokens.is_contiguous():
        raise ValueError(f"tokens: expected contiguous {tuple(s[:-1])}, got {tuple(tokens.shape)}")
    if ws.which != "states":
        raise ValueError("workspace: made for another call, expected a StatesWorkspace")
    if ws.buf.get_device() != index:
        raise ValueError(f"workspace: on {ws.buf.device}, tensors on {states.device}")
    return index, DTYPES[states.dtype], tokens.numel(), s[-1], stride, weight.shape[0], w[0]


def states_logprobs(states, weight, tokens, ws: StatesWorkspace, scale: float = 1.0,
                    flags: int = 0, stream=None) -> StatesLogprobs:
    """Log-probabilities of `tokens` ([T] or [B][T], -1: none), and log-sum-exp, of the logits
    scale * states @ weight.T: states [T][D] or [B][T][D] and weight [V][D], bf16 or f16, D a
    multiple of 8.  No logits are stored.  -logprob is the softmax cross entropy."""
    index, dtype, n, D, ss, V, wst = _rows(states, weight, tokens, ws)
    with made_on(stream, index):
        lp = torch.empty(tokens.shape, dtype=torch.float32, device=states.device)
        lse = torch.empty(tokens.shape, dtype=torch.float32, device=states.device)
    st = lib().sekv_states_logprobs(states.data_ptr(), dtype, n, D, ss, weight.data_ptr(), V, wst,
                                    tokens.data_ptr(), tokens.dtype == torch.int64, scale,
                                    lp.data_ptr(), lse.data_ptr(), flags, ws.buf.data_ptr(),
                                    ws.nbytes, raw_stream(stream, index))
    if st != 0:
        _check("sekv_states_logprobs", st)
    return StatesLogprobs(lp, lse)


def states_surprisal(states, weight, tokens, ws: StatesWorkspace, out=None, flags: int = 0,
                     stream=None):
    """H [B][T] f32 of the sequences `tokens` [B][T] with last states [B][T][D]: -log p of each
    token given those before it, 0 for the first; what build_spans takes."""
    if states.dim() != 3:
        raise ValueError(f"states: expected [B][T][D], got {tuple(states.shape)}")
    index, dtype, _, D, ss, V, wst = _rows(states, weight, tokens, ws)
    B, T = tokens.shape
    if out is None:
        with made_on(stream, index):
            out = torch.empty(B, T, dtype=torch.float32, device=states.device)
    else:
        check_tensor(out, "out", _F32, index)
        if out.shape != (B, T) or not out.is_contiguous():
            raise ValueError(f"out: expected contiguous [{B}][{T}], got {tuple(out.shape)}")
    st = lib().sekv_states_surprisal(states.data_ptr(), dtype, B, T, D, ss, weight.data_ptr(), V,
                                     wst, tokens.data_ptr(), tokens.dtype == torch.int64,
                                     out.data_ptr(), flags, ws.buf.data_ptr(), ws.nbytes,
                                     raw_stream(stream, index))
    if st != 0:
        _check("sekv_states_surprisal", st)
    return out


def _of_rows(t, name, tokens, index):
    if t is None:
        return None
    check_tensor(t, name, _F32, index)
    if t.shape != tokens.shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {tuple(tokens.shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _gradient(t, name, shape, dtype, index, device, stream):
    if t is None:
        with made_on(stream, index):
            return torch.empty(shape, dtype=dtype, device=device)
    check_tensor(t, name, (dtype,), index)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {tuple(shape)}, got {tuple(t.shape)}")
    return t


def states_logprobs_backward(states, weight, tokens, lse, grad, ws: StatesWorkspace,
                             grad_lse=None, scale: float = 1.0, want_states: bool = True,
                             want_weight: bool = True, d_states=None, d_weight=None,
                             flags: int = 0, stream=None):
    """(d_states, d_weight): the gradient of sum(grad * logprob) + sum(grad_lse * lse) by the
    arguments of states_logprobs, whose `lse` is given; grad and grad_lse f32 of tokens' shape
    (either may be None).  The mean cross entropy has grad = -1 / rows.  Gradients not wanted
    are None; given tensors (dense) are written."""
    index, dtype, n, D, ss, V, wst = _rows(states, weight, tokens, ws)
    p_lse = _of_rows(lse, "lse", tokens, index)
    p_grad = _of_rows(grad, "grad", tokens, index)
    p_grad_lse = _of_rows(grad_lse, "grad_lse", tokens, index)
    dx = dw = None
    if want_states:
        dx = _gradient(d_states, "d_states", states.shape, states.dtype, index, states.device, stream)
    if want_weight:
        dw = _gradient(d_weight, "d_weight", weight.shape, weight.dtype, index, states.device, stream)
    st = lib().sekv_states_logprobs_backward(
        states.data_ptr(), dtype, n, D, ss, weight.data_ptr(), V, wst, tokens.data_ptr(),
        tokens.dtype == torch.int64, scale, p_lse, p_grad, p_grad_lse,
        None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(), flags,
        ws.buf.data_ptr(), ws.nbytes, raw_stream(stream, index))
    if st != 0:
        _check("sekv_states_logprobs_backward", st)
    return dx, dw
