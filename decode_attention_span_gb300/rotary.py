"""Rotary positions (sekv_rope): argument marshalling only."""

from __future__ import annotations

import ctypes

import torch

from .sekv import DTYPES, _check, _ptr, _stream, check_tensor, lib

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3, "banded": 4}


class SekvRopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("original_context", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


class SekvHeads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("n_heads", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("x_stride", ctypes.c_int64 * 3),
                ("y_stride", ctypes.c_int64 * 3)]


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
        self._c = rope_config(rot_dim, base, interleaved, scaling, factor, original_context,
                              beta_fast, beta_slow, low_freq_factor, high_freq_factor,
                              attention_factor)
        freqs, self.mscale = rope_freqs(self._c)
        self.rot_dim = int(rot_dim)
        self.freqs = freqs.to(device or "cuda")


def _heads(x, y):
    xs, ys = x.stride(), y.stride()
    return SekvHeads(x.data_ptr(), y.data_ptr(), x.shape[2], 0, xs[:3], ys[:3])


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
    dev = x0.device
    B, T, _, D = x0.shape
    if D < plan.rot_dim:
        raise ValueError(f"rope: heads of {D} dimensions, plan rotates {plan.rot_dim}")
    if plan.freqs.device != dev:
        raise ValueError(f"plan: on {plan.freqs.device}, tensors on {dev}")
    check_tensor(positions, "positions", (torch.int32, torch.int64), dev)
    if positions.shape not in ((T,), (B, T)) or (T > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions: expected [{T}] or [{B}][{T}], got {tuple(positions.shape)}")
    heads = []
    outs = []
    for name, x, y in (("q", q, q_out), ("k", k, k_out)):
        if x is None:
            heads.append(None)
            outs.append(None)
            continue
        check_tensor(x, name, (x0.dtype,), dev)
        if x.dim() != 4 or x.shape[0] != B or x.shape[1] != T or x.shape[3] != D or x.stride(3) != 1:
            raise ValueError(f"{name}: expected [{B}][{T}][heads][{D}], got {tuple(x.shape)}")
        if y is None:
            y = torch.zeros_like(x, memory_format=torch.contiguous_format)
        else:
            check_tensor(y, name + "_out", (x0.dtype,), dev)
            if y.shape != x.shape or y.stride(3) != 1:
                raise ValueError(f"{name}_out: expected shape {tuple(x.shape)}, got {tuple(y.shape)}")
        heads.append(ctypes.byref(_heads(x, y)))
        outs.append(y)
    _check("sekv_rope",
           lib().sekv_rope(ctypes.byref(plan._c), plan.freqs.data_ptr(), plan.mscale,
                           DTYPES[x0.dtype], D, B, T, positions.data_ptr(),
                           positions.dtype == torch.int64,
                           positions.stride(0) if positions.dim() == 2 else 0, heads[0], heads[1],
                           1 if backward else 0, _stream(stream)))
    return outs[0], outs[1]
