"""Oracles of the token operators and the 4-bit cache against brute force and
closed forms, and the host-side refusals of their entry points (CPU)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import kv4, tokens


# ------------------------------------------------------------------ log-probabilities
def test_logprobs_of_every_token_sum_to_one_and_give_the_entropy():
    g = np.random.default_rng(0)
    x = g.normal(0, 3, (1, 40))
    lp = np.array([tokens.token_logprobs(x, [v], 0.7)["logprob"][0] for v in range(40)])
    r = tokens.token_logprobs(x, [3], 0.7, 40)
    assert abs(np.exp(lp).sum() - 1) < 1e-12
    assert abs(r["entropy"][0] + (np.exp(lp) * lp).sum()) < 1e-12
    assert np.allclose(r["top_logprobs"][0], -np.sort(-lp), atol=1e-12)
    assert np.array_equal(r["top_ids"][0], np.argsort(-lp, kind="stable"))


def test_logprobs_special_rows():
    inf = math.inf
    x = np.array([[0.0, 0, 0, 0], [-inf] * 4, [1.0, -inf, math.nan, 0], [0, inf, 0, 0], [2.0, -inf, 2, -inf]])
    r = tokens.token_logprobs(x, [-1, 2, 0, 0, 1], 1.0, 3)
    assert r["logprob"][0] == 0 and abs(r["entropy"][0] - math.log(4)) < 1e-15
    assert list(r["top_ids"][0]) == [0, 1, 2]
    assert r["logprob"][1] == -inf and r["lse"][1] == -inf and r["entropy"][1] == 0
    assert np.isnan(r["logprob"][2:4]).all() and np.isnan(r["entropy"][2:4]).all()
    assert r["logprob"][4] == -inf and list(r["top_ids"][4]) == [0, 2, -1]


def test_surprisal_is_shifted():
    x = np.zeros((2, 3, 8))
    x[0, 0, 5] = 100.0
    H = tokens.surprisal(x, np.array([[1, 5, 2], [0, 0, 0]]))
    assert H[0, 0] == 0 and abs(H[0, 1]) < 1e-12 and abs(H[0, 2] - math.log(8)) < 1e-12
    assert np.allclose(H[1], [0, math.log(8), math.log(8)])


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("inter", [False, True])
def test_rope_dot_products_depend_on_the_distance_alone(inter):
    g = np.random.default_rng(1)
    f, _ = tokens.rope_frequencies(16, 10000.0)
    q, k = g.normal(size=(1, 1, 1, 24)), g.normal(size=(1, 1, 1, 24))
    dot = lambda a, b: float((tokens.rope(q, [[a]], f, 1.0, inter) * tokens.rope(k, [[b]], f, 1.0, inter)).sum())  # noqa: E731
    assert abs(dot(7, 3) - dot(1007, 1003)) < 1e-10
    back = tokens.rope(tokens.rope(q, [[99]], f, 1.0, inter), [[99]], f, 1.0, inter, backward=True)
    assert np.allclose(back, q, atol=1e-13)
    assert np.array_equal(tokens.rope(q, [[5]], f, 1.0, inter)[..., 16:], q[..., 16:])
    assert np.array_equal(tokens.rope(q, [[-1]], f, 1.0, inter), q)


def test_rope_scalings_closed_forms():
    u, _ = tokens.rope_frequencies(64, 10000.0)
    assert np.allclose(u, 10000.0 ** (-np.arange(32) / 32))
    assert np.allclose(tokens.rope_frequencies(64, 10000.0, "linear", 4.0)[0], u / 4)
    ntk = tokens.rope_frequencies(64, 10000.0, "ntk", 4.0)[0]
    assert abs(ntk[0] - 1) < 1e-15 and abs(ntk[-1] - u[-1] / 4) < 1e-12 * u[-1]
    for kind in ("parts", "banded"):  # fast pairs keep their pace, slow ones are stretched in full
        s, m = tokens.rope_frequencies(64, 10000.0, kind, 4.0, 4096)
        assert s[0] == u[0] and abs(s[-1] - u[-1] / 4) < 1e-18
        assert np.all((s <= u * (1 + 1e-15)) & (s >= u / 4 * (1 - 1e-15)))
        assert abs(m - (0.1 * math.log(4) + 1 if kind == "parts" else 1)) < 1e-15


def test_rope_table_is_the_frequencies_as_turns(libsekv):
    from decode_attention_span_gb300 import rotary
    for rot, base, kind, factor in ((128, 500000.0, "banded", 8.0), (64, 1e4, "parts", 16.0),
                                    (2, 1e4, "none", 1.0), (96, 1e6, "ntk", 4.0),
                                    (32, 1e4, "linear", 0.125)):
        freqs, m = rotary.rope_freqs(rotary.rope_config(rot, base, scaling=kind, factor=factor))
        f, mo = tokens.rope_frequencies(rot, base, kind, factor)
        turns = freqs.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
        # pow, exp and the division err by a few 2^-53 of the value each
        assert np.allclose(turns, np.mod(f / (2 * math.pi), 1.0), rtol=2 ** -46, atol=2 ** -60)
        assert abs(m - mo) <= 2 ** -23 * mo


# ------------------------------------------------------------------ the 4-bit cache
def test_kv4_layout_uses_every_nibble_once():
    seen = set()
    for j in range(16):
        for d in range(128):
            for f in (kv4.k_byte, kv4.v_byte):
                seen.add((f(j, d), d % 2))
        for g in range(2):
            for v in (0, 1):
                seen |= {(kv4.param_byte(j, g, v) + i, n) for i in range(4) for n in range(2)}
    assert seen == {(b, n) for b in range(2304) for n in range(2)}


def test_kv4_quantise_error_and_edges():
    g = np.random.default_rng(2)
    x = kv4.bf16_value(kv4.bf16_bits(g.normal(0, 2, (50, 128)) + g.normal(0, 5, (50, 1))))
    n, sb, zb = kv4.quantise(x)
    y = kv4.values(n, sb, zb)
    s = np.repeat(kv4.bf16_value(sb), 64, -1)
    # half a step, and what rounding s (2^-9) takes off the top of the range
    assert np.all(np.abs(y - x) <= s * (0.5 + 15 * 2.0 ** -8))
    flat = np.full((1, 128), 3.5, np.float32)
    flat[0, 64:] = -1e38
    n, sb, zb = kv4.quantise(flat)
    # a constant that is a bf16 value is its own zero point; one that is not sits at the top of a step
    assert not n[0, :64].any() and sb[0, 0] == 0 and (kv4.values(n, sb, zb)[0, :64] == 3.5).all()
    assert (n[0, 64:] == 15).all() and np.allclose(kv4.values(n, sb, zb)[0, 64:], -1e38, rtol=2.0 ** -15)
    bad = np.zeros((3, 128), np.float32)
    bad[0, 3], bad[1, 70], bad[2, 0], bad[2, 1] = math.nan, math.inf, 3e38, -3e38
    n, sb, zb = kv4.quantise(bad)
    y = kv4.values(n, sb, zb)
    assert np.isnan(y[0, :64]).all() and not y[0, 64:].any()
    assert np.isnan(y[1, 64:]).all() and not y[1, :64].any()
    assert np.isnan(y[2, :64]).all()


def test_kv4_put_get_and_attention_against_dense_softmax():
    g = np.random.default_rng(3)
    B, H, T = 2, 2, 70
    pages = g.integers(0, 256, (6, H, kv4.PAGE_BYTES)).astype(np.uint8)
    table = np.array([[4, 1], [2, 5]])
    ref = np.zeros((2, B, H, T, 128))
    for b in range(B):
        for c in range(H):
            for t in range(T):
                for v in (0, 1):
                    n, sb, zb = kv4.quantise(g.normal(size=128))
                    kv4.put(pages, table, b, c, t, n, sb, zb, v)
                    ref[v, b, c, t] = kv4.values(n, sb, zb)
    q = g.normal(size=(B, 2, 4, 128))
    out, lse, _, _ = kv4.attention(q, pages, table, [70, 1], 0.1)
    for i in range(2):
        for h in range(4):
            K, V = ref[0, 0, h // 2][:69 + i], ref[1, 0, h // 2][:69 + i]
            p = np.exp(K @ q[0, i, h] * 0.1)
            assert np.allclose(out[0, i, h], p @ V / p.sum(), atol=1e-12)
            assert abs(lse[0, i, h] - math.log(p.sum())) < 1e-12
    assert not out[1, 0].any() and (lse[1, 0] == -math.inf).all()  # one token, two queries
    assert np.allclose(out[1, 1, 2], ref[1, 1, 1, 0])


# ------------------------------------------------------------------ host-side refusals
@pytest.fixture(scope="module")
def libsekv():
    from decode_attention_span_gb300 import build, sekv
    build.build()
    return sekv.lib()


P = ctypes.c_void_p(1 << 20)   # an aligned address that no call here dereferences
ODD = ctypes.c_void_p((1 << 20) + 1)
INVALID, CAPACITY, UNSUPPORTED = -1, -2, -5


def test_logprobs_refusals(libsekv):
    def call(logits=P, dtype=0, batch=1, n=4, vocab=100, tok=P, scale=1.0, top=0, lp=P, ids=None, tlp=None, ws=P, nb=4096):
        return libsekv.sekv_token_logprobs(logits, dtype, batch, n, vocab, 0, vocab, tok, 0, 0, scale, top, lp, None, None, ids, tlp, ws, nb, None)
    assert call(n=0) == 0 and call(batch=0) == 0
    for kw in (dict(logits=None), dict(logits=ODD), dict(dtype=3), dict(dtype=-1), dict(batch=-1), dict(n=-1),
               dict(vocab=0), dict(tok=None), dict(tok=ODD), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
               dict(scale=math.nan), dict(top=-1), dict(lp=None), dict(top=2), dict(top=2, ids=P), dict(ids=P, tlp=P),
               dict(ws=None)):
        assert call(**kw) == INVALID, kw
    assert call(nb=8) == CAPACITY
    assert call(top=33, ids=P, tlp=P) == UNSUPPORTED
    assert call(vocab=(1 << 30) + 1) == UNSUPPORTED and call(n=1 << 31) == UNSUPPORTED
    assert libsekv.sekv_surprisal(P, 0, 1, 4, 10, 0, 10, P, 0, 0, None, P, 4096, None) == INVALID
    assert libsekv.sekv_surprisal(P, 0, 1, 0, 10, 0, 10, P, 0, 0, P, P, 4096, None) == 0


def test_rope_refusals(libsekv):
    from decode_attention_span_gb300 import rotary

    def table(**kw):
        buf = (ctypes.c_uint64 * 256)()
        m = ctypes.c_float()
        return libsekv.sekv_rope_freqs(ctypes.byref(rotary.rope_config(**{"rot_dim": 64, **kw})), buf, ctypes.byref(m))
    assert table() == 0
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=math.inf), dict(scaling="linear", factor=0.0),
               dict(scaling="parts", original_context=0), dict(scaling="parts", beta_fast=0.0),
               dict(scaling="banded", low_freq_factor=4.0), dict(rot_dim=2, scaling="ntk", factor=2.0),
               dict(attention_factor=-1.0), dict(attention_factor=math.nan)):
        assert table(**kw) == INVALID, kw
    assert table(rot_dim=514) == UNSUPPORTED
    with pytest.raises(ValueError):
        rotary.rope_config(64, scaling="other")

    heads = lambda x=1 << 20, y=1 << 21, n=2, xs=(0, 256, 128), ys=(0, 256, 128): ctypes.byref(  # noqa: E731
        rotary.SekvHeads(x or 0, y, n % (1 << 32), *xs, *ys))

    def call(dtype=0, dim=128, B=1, T=2, pos=P, q=heads(), k=None, flags=0, m=1.0, freqs=P):
        return libsekv.sekv_rope(ctypes.byref(rotary.rope_config(64)), freqs, m, dtype, dim, B, T, pos, 0, 0, q, k, flags, None)
    assert call(T=0) == 0 and call(q=heads(n=0)) == 0
    for kw in (dict(dtype=5), dict(dim=62), dict(B=-1), dict(pos=None), dict(pos=ODD), dict(q=None), dict(flags=2),
               dict(m=math.nan), dict(freqs=None), dict(q=heads(x=None)), dict(q=heads(x=(1 << 20) + 1)), dict(q=heads(n=-1)),
               dict(q=heads(y=1 << 20, ys=(0, 128, 256)))):
        assert call(**kw) == INVALID, kw
    # output rows on one another, which a broadcast tensor given for the output has
    for kw in (dict(q=heads(ys=(0, 256, 0))), dict(q=heads(ys=(0, 0, 128))), dict(B=2), dict(k=heads(ys=(512, 0, 128))),
               dict(q=heads(y=1 << 20, xs=(0, 0, 128), ys=(0, 0, 128)))):
        assert call(**kw) == INVALID, kw
    assert call(dim=1026) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED and call(q=heads(n=65535), k=heads(n=1)) == UNSUPPORTED


def test_kv4_refusals(libsekv):
    import decode_attention_span_gb300 as sk
    from decode_attention_span_gb300.kv4 import SekvKv4Cache
    S = (ctypes.c_int64 * 3)(8, 8, 8)

    def args(cfg=(1, 8, 2), cache=(1 << 20, 1 << 20, 4, 4)):
        return ctypes.byref(sk.Config(*cfg, 0, 0, 64).c()), None if cache is None else ctypes.byref(SekvKv4Cache(*cache))
    append = lambda a=args(), dt=0, k=P, ks=S, n=1, first=P, ws=P: libsekv.sekv_kv4_append(  # noqa: E731
        *a, dt, k, ks, P, S, n, first, None, ws, 0, None)
    read = lambda a=args(), dt=0, k=P, n=1, ws=P: libsekv.sekv_kv4_read(*a, dt, k, P, n, P, None, ws, 0, None)  # noqa: E731
    attn = lambda a=args(), dt=0, q=P, nq=1, ws=P, scale=1.0: libsekv.sekv_kv4_attention(  # noqa: E731
        *a, dt, q, nq, P, scale, P, P, ws, 0, None)
    for f in (append, read, attn):
        assert f(args(cfg=(1025, 8, 2))) == UNSUPPORTED
        assert f(args(cfg=(1, 18, 2))) == UNSUPPORTED and f(args(cfg=(1, 7, 2))) == INVALID
        assert f(args(cache=None)) == INVALID and f(ws=None) == INVALID and f(ws=ODD) == INVALID
        for bad in ((None, 1 << 20, 4, 4), (1 << 20, None, 4, 4), ((1 << 20) + 8, 1 << 20, 4, 4), (1 << 20, 1 << 20, 0, 4), (1 << 20, 1 << 20, 4, 0)):
            assert f(args(cache=bad)) == INVALID, bad
        assert f(a=(None, args()[1])) == INVALID
    for nq in (0, -1, 65):
        assert attn(nq=nq) == UNSUPPORTED
    assert attn(args(cache=(1 << 20, 1 << 20, 4, 1 << 24))) == UNSUPPORTED
    assert attn(args(cfg=(1024, 512, 512), cache=(1 << 20, 1 << 20, 4, 1 << 10))) == UNSUPPORTED
    # what does not depend on the GPU's size is refused before the workspace is looked at
    for f, kw in ((append, dict(dt=2)), (append, dict(k=None)), (append, dict(k=ODD)), (append, dict(n=-1)), (append, dict(first=None)),
                  (append, dict(ks=(ctypes.c_int64 * 3)(8, 8, 4))), (append, dict(n=2, ks=(ctypes.c_int64 * 3)(8, 4, 8))), (read, dict(dt=3)), (read, dict(k=None)), (read, dict(n=-1)),
                  (attn, dict(dt=2)), (attn, dict(q=None)), (attn, dict(q=ODD)), (attn, dict(scale=math.nan)),
                  (attn, dict(scale=0.0)), (attn, dict(scale=-0.1)), (attn, dict(scale=math.inf))):
        assert f(**kw) == INVALID, kw


def test_binding_refuses_tensors_off_the_gpu(libsekv):
    import torch
    import decode_attention_span_gb300 as sk

    class NoWs:
        buf = torch.empty(64, dtype=torch.uint8)
        nbytes = 64
        ptr = staticmethod(lambda: None)
    with pytest.raises(ValueError):
        sk.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), NoWs)
    with pytest.raises(TypeError):
        sk.token_logprobs(torch.zeros(2, 8, dtype=torch.float64), torch.zeros(2, dtype=torch.int64), NoWs)
    cfg = sk.Config(1, 2, 1, 0, 0, 64)
    with pytest.raises(ValueError):
        sk.Kv4Cache(cfg, torch.empty(2, 1, 9216, dtype=torch.uint8), torch.zeros(1, 2, dtype=torch.int32))
    plan = sk.RopePlan(8, device="cpu")
    with pytest.raises(ValueError):
        sk.rope(plan, torch.zeros(1, 2, 1, 8), None, torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sk.rope(plan, None, None, torch.zeros(2, dtype=torch.int32))
