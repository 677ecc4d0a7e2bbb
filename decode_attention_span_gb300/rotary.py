"""Rotary positions (sekv_rope): argument marshalling only."""

from __future__ import annotations

import ctypes

import torch

from .sekv import DTYPES, _check, _ptr, check_tensor, current_index, lib, made_on, raw_stream

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3, "banded": 4}


class SekvRopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("original_context", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


# sekv_heads as nine 64-bit words: x, y, n_heads | zero_padding << 32, strides of x and of y
SekvHeads = ctypes.c_int64 * 9


def rope_config(rot_dim: int, base: float = 10000.0, interleaved: bool = False,
                scaling: str = "none", factor: float = 1.0, original_context: int = 8192,
                beta_fast: float = 32.0, beta_slow: float = 1.0, low_freq_factor: float = 1.0,
                high_freq_factor: float = 4.0, attention_factor: float = 0.0) -> SekvRopeConfig:
    if scaling not in SCALINGS:
        raise ValueError(f"scaling: one of {sorted(SCALINGS)}, got {scaling!r}")
    return SekvRopeConfig(int(rot_dim), int(interleaved), SCALINGS[scaling],
                          int(original_context), base, factor, beta_fast, beta_slow,
                          low_freq_factor, high_freq_factor, attention_factor)


def rope_freqs(config: SekvRopeConfig):
    """sekv_rope_freqs: (turns per position of each pair as 64-bit fixed-point
    fractions, in a host int64 tensor; the factor on the result)."""
    n = max(config.rot_dim // 2, 1)
    freqs = torch.empty(n, dtype=torch.int64)
    m = ctypes.c_float(0.0)
    _check("sekv_rope_freqs", lib().sekv_rope_freqs(ctypes.byref(config), _ptr(freqs),
                                                    ctypes.byref(m)))
    return freqs, m.value


class RopePlan:
    """Frequencies of a rotary embedding on the device, made once and kept.

    rot_dim    leading dimensions of a head that turn (even)
    scaling    "none", "linear", "ntk", "parts" (ramp between the pairs that turn
               beta_fast and beta_slow times in original_context) or "banded" (between
               low_freq_factor and high_freq_factor turns); formulas in include/sekv.h
    """

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_context: int = 8192,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, low_freq_factor: float = 1.0,
                 high_freq_factor: float = 4.0, attention_factor: float = 0.0, device=None):
        config = rope_config(rot_dim, base, interleaved, scaling, factor, original_context,
                             beta_fast, beta_slow, low_freq_factor, high_freq_factor,
                             attention_factor)
        freqs, self.mscale = rope_freqs(config)
        self.config, self._c = config, ctypes.byref(config)
        self.rot_dim = int(rot_dim)
        self.freqs = freqs.to(device or "cuda")
        self.freqs_ptr, self.device_index = self.freqs.data_ptr(), self.freqs.get_device()


_POSITIONS = (torch.int32, torch.int64)


def _heads(name, x, y, B, T, D, dtype, index, stream):
    """(sekv_heads, output) of one tensor; an output made here is zero at padding."""
    if x.dtype != dtype or x.get_device() != index:
        check_tensor(x, name, (dtype,), index)
    s, xs = x.shape, x.stride()
    if len(s) != 4 or s[0] != B or s[1] != T or s[3] != D or xs[3] != 1:
        raise ValueError(f"{name}: expected [{B}][{T}][heads][{D}] with consecutive elements in a "
                         f"head, got {tuple(s)}")
    n = s[2]
    if y is None:
        with made_on(stream, index):
            y = torch.empty_like(x, memory_format=torch.contiguous_format)
        return SekvHeads(x.data_ptr(), y.data_ptr(), n + (1 << 32), xs[0], xs[1], xs[2],
                         T * n * D, n * D, D), y
    if y.dtype != dtype or y.get_device() != index:
        check_tensor(y, name + "_out", (dtype,), index)
    ys = y.stride()
    if y.shape != s or ys[3] != 1:
        raise ValueError(f"{name}_out: expected shape {tuple(s)}, got {tuple(y.shape)}")
    return SekvHeads(x.data_ptr(), y.data_ptr(), n, xs[0], xs[1], xs[2], ys[0], ys[1], ys[2]), y


def rope(plan: RopePlan, q, k, positions, q_out=None, k_out=None, backward: bool = False,
         stream=None):
    """Rotates q [B][T][Hq][D] and k [B][T][Hkv][D] (either may be None) to the
    positions [B][T] or [T] of their tokens; returns (q_out, k_out).

    Inputs and outputs may have any strides with the last one 1, so that
    ``k_out=K.transpose(1, 2)`` writes the [B][Hkv][T][D] layout of the span build, and
    ``q_out=q`` rotates in place.  A token with a negative position is neither
    read nor written (outputs made here are zero there).  backward=True turns the
    other way: the gradient, and for a plan without a factor the inverse."""
    x0 = q if q is not None else k
    if x0 is None:
        raise ValueError("rope: q or k is needed")
    dtype = x0.dtype
    code = DTYPES.get(dtype)
    if code is None or x0.dim() != 4:
        raise TypeError(f"rope: expected [B][T][heads][D] of {list(DTYPES)}, got {dtype} "
                        f"{tuple(x0.shape)}")
    index = current_index(x0, "rope")
    B, T, _, D = x0.shape
    if D < plan.rot_dim:
        raise ValueError(f"rope: heads of {D} dimensions, plan rotates {plan.rot_dim}")
    if plan.device_index != index:
        raise ValueError(f"plan: on {plan.freqs.device}, tensors on {x0.device}")
    check_tensor(positions, "positions", _POSITIONS, index)
    s, ps = positions.shape, positions.stride()
    if len(s) == 2 and s[0] == B and s[1] == T:
        pos_stride = ps[0]
    elif len(s) == 1 and s[0] == T:
        pos_stride = 0
    else:
        raise ValueError(f"positions: expected [{T}] or [{B}][{T}], got {tuple(s)}")
    if T > 1 and ps[-1] != 1:
        raise ValueError("positions: must be consecutive along a sequence")
    qh = kh = None
    if q is not None:
        qh, q_out = _heads("q", q, q_out, B, T, D, dtype, index, stream)
    if k is not None:
        kh, k_out = _heads("k", k, k_out, B, T, D, dtype, index, stream)
    st = lib().sekv_rope(plan._c, plan.freqs_ptr, plan.mscale, code, D, B, T,
                         positions.data_ptr(), positions.dtype == torch.int64, pos_stride, qh, kh,
                         1 if backward else 0, raw_stream(stream, index))
    if st != 0:
        _check("sekv_rope", st)
    return q_out, k_out
