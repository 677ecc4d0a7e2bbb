"""Plain form of the 4-bit cache: quantisation, page layout, attention.  The
layout is written out index by index from the C header; shares nothing with the
CUDA path."""

from __future__ import annotations

import math

import numpy as np

PAGE_BYTES = 9216


def bf16_bits(x):
    """Bits of fp32 values rounded to bf16, to nearest even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, np.uint32) << 16).view(np.float32)


def bf16_floor_bits(x):
    """Bits of the largest bf16 at or below each finite fp32 value."""
    u = np.asarray(x, np.float32).view(np.uint32)
    up = (u >> 31 == 1) & (u & 0xFFFF != 0)  # negative and inexact: away from zero
    return ((u >> 16) + up).astype(np.uint16)


def quantise(x):
    """x [..., 128] -> (codes uint8 [..., 128], s and z as bf16 bits [..., 2])."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], 2, 64)
    ok = np.isfinite(g).all(-1)
    g0 = np.where(ok[..., None], g, np.float32(0))
    zb = bf16_floor_bits(g0.min(-1))
    z = bf16_value(zb)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        q = (g0.max(-1) - z) * np.float32(1 / 15)
        sb = bf16_bits(q)
        s = bf16_value(sb)
        n = np.where(s[..., None] > 0, (g0 - z[..., None]) / s[..., None], np.float32(0))
        n = np.clip(np.rint(n), 0, 15)
    ok &= np.isfinite(s)
    zb = np.where(ok, zb, 0x7FFF).astype(np.uint16)
    sb = np.where(ok, sb, 0x7FFF).astype(np.uint16)
    return np.where(ok[..., None], n, 0).astype(np.uint8).reshape(x.shape), sb, zb


def values(codes, sb, zb):
    """What codes stand for, fp64 [..., 128]."""
    s, z = bf16_value(sb).astype(np.float64), bf16_value(zb).astype(np.float64)
    n = codes.reshape(*codes.shape[:-1], 2, 64)
    return (z[..., None] + s[..., None] * n).reshape(codes.shape)


def k_byte(j, d):
    return 64 * j + 16 * ((d % 64) // 16) + 8 * (d // 64) + (d % 16) // 2


def v_byte(j, d):
    e, u, o = 8 * (j // 8), (j % 8) // 2, j % 2
    return 1024 + 64 * e + 64 * ((d % 64) // 8) + 16 * u + 8 * (d // 64) + 4 * ((d % 8) // 4) + 2 * o + (d % 4) // 2


def param_byte(j, g, is_v):
    e, u, o = 8 * (j // 8), (j % 8) // 2, j % 2
    return 2048 + 128 * is_v + 32 * u + 2 * e + 8 * o + 4 * g


def put(pages, table, b, c, t, codes, sb, zb, is_v):
    """Writes one token's K or V (codes [128], bits [2]) into pages [P][Hkv][9216]."""
    page = pages[int(table[b][t // 64]), c]
    tile = page[(t % 64) // 16 * 2304:][:2304]
    j = t % 16
    for d in range(128):
        at = v_byte(j, d) if is_v else k_byte(j, d)
        old = int(tile[at])
        tile[at] = (old & 0x0F) | int(codes[d]) << 4 if d % 2 else (old & 0xF0) | int(codes[d])
    for g in range(2):
        at = param_byte(j, g, is_v)
        tile[at:at + 2] = np.frombuffer(np.uint16(sb[g]).tobytes(), np.uint8)
        tile[at + 2:at + 4] = np.frombuffer(np.uint16(zb[g]).tobytes(), np.uint8)


def get(pages, table, b, c, n):
    """K and V fp64 [n][128] of the first n tokens of sequence b, KV head c, and the fp64
    magnitudes |z| + 15 |s| of their groups [n][2] each."""
    d = np.arange(128)
    out = []
    for is_v in (False, True):
        byte = np.array([[(v_byte if is_v else k_byte)(j, int(i)) for i in d] for j in range(16)])
        t = np.arange(n)
        page = np.asarray(table[b], np.int64)[t // 64]
        flat = pages[page, c].reshape(n, 4, 2304)[np.arange(n), (t % 64) // 16] if n else np.zeros((0, 2304), np.uint8)
        code = (flat[np.arange(n)[:, None], byte[t % 16]] >> (4 * (d % 2))) & 15
        p = np.array([[param_byte(j, g, is_v) for g in range(2)] for j in range(16)]).reshape(16, 2)[t % 16]
        word = lambda off: (flat[np.arange(n)[:, None], p + off].astype(np.uint16)  # noqa: E731
                            | flat[np.arange(n)[:, None], p + off + 1].astype(np.uint16) << 8)
        sb, zb = word(0), word(2)
        out.append(values(code, sb, zb))
        out.append(np.abs(bf16_value(zb).astype(np.float64)) + 15 * np.abs(bf16_value(sb).astype(np.float64)))
    return out[0], out[2], out[1], out[3]


def attention(q, pages, table, lens, scale):
    """q [B][n_q][Hq][128] fp64 -> (out, lse, bound): bound is what an error of one part in
    one of the weights, or of one in a logit, can move each output by at most (the weighted
    mean of the values' largest parts)."""
    B, nq, Hq, _ = q.shape
    Hkv = pages.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -math.inf)
    bound = np.zeros(q.shape)
    logit = np.zeros(q.shape[:3])  # scale of the terms a logit is summed from
    for b in range(B):
        for c in range(Hkv):
            K, V, ka, va = get(pages, table, b, c, int(lens[b]))
            for i in range(nq):
                n = int(lens[b]) - (nq - 1 - i)
                if n <= 0:
                    continue
                for h in range(c * G, c * G + G):
                    x = K[:n] @ q[b, i, h] * scale
                    m = x.max()
                    e = np.exp(x - m)
                    p = e / e.sum()
                    out[b, i, h] = p @ V[:n]
                    lse[b, i, h] = m + math.log(e.sum())
                    bound[b, i, h] = np.repeat(p @ va[:n], 64)
                    logit[b, i, h] = abs(scale) * np.abs(q[b, i, h]).sum() * ka[:n].max()
    return out, lse, bound, logit
