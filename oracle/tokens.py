"""Plain fp64 forms of the token operators: log-probabilities with entropy and
alternatives, surprisal, rotary positions.  Written from the formulas in the
C header; pinned by tests/test_oracle_operators.py against brute force and
closed forms."""

from __future__ import annotations

import math

import numpy as np


def token_logprobs(logits, tokens, scale=1.0, n_top=0):
    """logits [R][V] (any float array), tokens [R] -> dict of fp64 arrays (ids int32),
    with the header's conventions for -1, -inf rows, NaN and +inf."""
    x = np.asarray(logits, np.float64)
    R, V = x.shape
    lp, lse, ent = np.zeros(R), np.zeros(R), np.zeros(R)
    ids = np.full((R, n_top), -1, np.int32)
    tlp = np.full((R, n_top), -math.inf)
    for r in range(R):
        row, tok = x[r], int(tokens[r])
        if np.isnan(row).any() or (row == math.inf).any():
            lp[r] = lse[r] = ent[r] = math.nan
            tlp[r] = math.nan
            continue
        m = row.max()
        if m == -math.inf:
            lse[r], ent[r] = -math.inf, 0.0
            lp[r] = 0.0 if tok == -1 else -math.inf
        else:
            d = (row - m) * scale
            e = np.exp(d)
            S = e.sum()
            d0 = np.where(np.isfinite(d), d, 0.0)
            lse[r], ent[r] = scale * m + math.log(S), math.log(S) - (e * d0).sum() / S
            lp[r] = 0.0 if tok == -1 else (d[tok] - math.log(S) if 0 <= tok < V else math.nan)
            order = np.lexsort((np.arange(V), -(row + 0.0)))[:n_top]
            order = order[row[order] > -math.inf]
            ids[r, :len(order)] = order
            tlp[r, :len(order)] = d[order] - math.log(S)
        if tok != -1 and not 0 <= tok < V:
            lp[r] = math.nan
    return dict(logprob=lp, lse=lse, entropy=ent, top_ids=ids, top_logprobs=tlp)


def surprisal(logits, tokens):
    """logits [B][T][V], tokens [B][T] -> H [B][T]."""
    B, T, _ = logits.shape
    H = np.zeros((B, T))
    for b in range(B):
        if T > 1:
            H[b, 1:] = -token_logprobs(logits[b, :-1], tokens[b, 1:])["logprob"]
    return H + 0.0


def states_logprobs(states, weight, tokens, scale=1.0):
    """states [R][D], weight [V][D] -> dict(logprob, lse) of the logits scale * states @ weight.T."""
    r = token_logprobs(np.asarray(states, np.float64) @ np.asarray(weight, np.float64).T * scale, tokens)
    return dict(logprob=r["logprob"], lse=r["lse"])


def states_gradient(states, weight, tokens, grad, grad_lse, scale=1.0):
    """(d_states, d_weight, G) of sum(grad * logprob) + sum(grad_lse * lse): logprob of token -1 is
    0, whatever the states."""
    h, w = np.asarray(states, np.float64), np.asarray(weight, np.float64)
    x = h @ w.T * scale
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    G = grad_lse[:, None] * p
    for r, t in enumerate(tokens):
        if t >= 0:
            G[r] -= grad[r] * p[r]
            G[r, t] += grad[r]
    G *= scale
    return G @ w, G.T @ h, G


def rope_frequencies(rot, base, scaling="none", factor=1.0, original=8192, beta_fast=32.0,
                     beta_slow=1.0, low=1.0, high=4.0, attention_factor=0.0):
    """(angle per position of each pair, factor on the result)."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        u = b ** (-2.0 * i / rot)
        if scaling == "linear":
            u /= factor
        if scaling == "parts":
            pair = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(0, math.floor(pair(beta_fast))), min(rot - 1, math.ceil(pair(beta_slow)))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            u = (1 - r) * u + r * u / factor
        if scaling == "banded":
            s = min(1.0, max(0.0, (original * u / (2 * math.pi) - low) / (high - low)))
            u = (1 - s) * u / factor + s * u
        out.append(u)
    m = 0.1 * math.log(factor) + 1.0 if scaling == "parts" and factor > 1 else 1.0
    return np.array(out), attention_factor or m


def rope(x, positions, freqs, mscale=1.0, interleaved=False, backward=False):
    """x [B][T][H][D], positions [B][T]; tokens at negative positions come back as they are."""
    y = np.array(x, np.float64)
    n = len(freqs)
    for b in range(y.shape[0]):
        for t in range(y.shape[1]):
            p = int(positions[b][t])
            if p < 0:
                continue
            ang = p * freqs * (-1.0 if backward else 1.0)
            c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
            ia = np.arange(n) * 2 if interleaved else np.arange(n)
            ib = ia + 1 if interleaved else ia + n
            a, q = y[b, t][:, ia].copy(), y[b, t][:, ib].copy()
            y[b, t][:, ia] = a * c - q * s
            y[b, t][:, ib] = q * c + a * s
    return y
