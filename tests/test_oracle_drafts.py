"""CPU: the oracles of tree attention, of keeping a branch and of log-probabilities from states, pinned
against closed forms and differences; refusals of the calls on the host."""
import ctypes
import math

import numpy as np
import pytest

from oracle import kv4, tokens


@pytest.fixture(scope="module")
def libsekv():
    from decode_attention_span_gb300 import build, sekv
    build.build()
    return sekv.lib()


P, ODD, INVALID, UNSUPPORTED = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8), -1, -5


def small_cache(n, H=1, seed=0):
    rng = np.random.default_rng(seed)
    mp = -(-n // 64)
    pages = rng.integers(0, 256, (mp + 1, H, 9216), dtype=np.uint8)
    table = rng.permutation(mp + 1)[:mp][None].astype(np.int32)
    for c in range(H):
        for t in range(n):
            x = rng.normal(size=(2, 128))
            for v in range(2):
                codes, sb, zb = kv4.quantise(x[v].astype(np.float32))
                kv4.put(pages, table, 0, c, t, codes, sb, zb, bool(v))
    return pages, table


# ------------------------------------------------------------------ trees
def test_a_chain_is_the_attention_of_the_last_tokens():
    pages, table = small_cache(70, 2)
    q = np.random.default_rng(1).normal(size=(1, 5, 4, 128))
    tree = [[(1 << (i + 1)) - 1 for i in range(5)]]
    got = kv4.tree_attention(q, pages, table, [65], tree, 0.09)
    want = kv4.attention(q, pages, table, [70], 0.09)
    for g, w in zip(got, want):
        assert np.allclose(g, w, rtol=1e-12, atol=0)


def test_siblings_do_not_see_each_other_and_empty_masks_give_nothing():
    pages, table = small_cache(4)
    q = np.random.default_rng(2).normal(size=(1, 4, 1, 128))
    # no prefix: token 1 sees itself alone, token 2 nothing, token 3 sees 0 and itself
    out, lse, _, _ = kv4.tree_attention(q, pages, table, [0], [[1, 2, 0, 9]], 0.1)
    K, V, _, _ = kv4.get(pages, table, 0, 0, 4)
    assert np.allclose(out[0, 1, 0], V[1]) and np.isclose(lse[0, 1, 0], K[1] @ q[0, 1, 0] * 0.1)
    assert not out[0, 2].any() and lse[0, 2, 0] == -math.inf
    x = K[[0, 3]] @ q[0, 3, 0] * 0.1
    p = 1 / (1 + math.exp(x[1] - x[0]))
    assert np.allclose(out[0, 3, 0], p * V[0] + (1 - p) * V[3])
    # a negative first: the sequence's tokens see nothing
    out, lse, _, _ = kv4.tree_attention(q, pages, table, [-2], [[1, 3, 7, 15]], 0.1)
    assert not out.any() and (lse == -math.inf).all()


def test_kept_tokens_read_as_they_did():
    pages, table = small_cache(80)
    before = kv4.get(pages, table, 0, 0, 80)
    kv4.keep(pages, table, 0, 0, 60, [1, 2, 7, 19])
    after = kv4.get(pages, table, 0, 0, 80)
    for x, y in zip(before, after):
        assert np.array_equal(y[:60], x[:60])
        assert np.array_equal(y[60:64], x[[61, 62, 67, 79]])
        assert np.array_equal(y[64:], x[64:])


# ------------------------------------------------------------------ states
def test_gradient_of_states_against_differences():
    rng = np.random.default_rng(3)
    h, w = rng.normal(size=(4, 6)), rng.normal(size=(9, 6))
    tok, g, e = [2, -1, 8, 2], rng.normal(size=4), rng.normal(size=4)

    def value(h, w):
        r = tokens.states_logprobs(h, w, tok, 0.7)
        return (g * r["logprob"]).sum() + (e * r["lse"]).sum()
    dh, dw, _ = tokens.states_gradient(h, w, tok, g, e, 0.7)
    for x, d in ((h, dh), (w, dw)):
        for i in np.ndindex(x.shape):
            old, step = x[i], 1e-5
            x[i] = old + step
            up = value(h, w)
            x[i] = old - step
            down = value(h, w)
            x[i] = old
            assert abs((up - down) / (2 * step) - d[i]) < 1e-8


def test_gradient_sums_to_nothing_over_the_vocabulary():
    rng = np.random.default_rng(4)
    h, w = rng.normal(size=(3, 5)), rng.normal(size=(7, 5))
    _, _, G = tokens.states_gradient(h, w, [0, 6, 3], np.ones(3), np.zeros(3))
    assert np.allclose(G.sum(1), 0, atol=1e-15) and (G[[0, 1, 2], [0, 6, 3]] > 0).all()


# ------------------------------------------------------------------ refusals
def cache_args(cfg=(1, 8, 2), cache=(1 << 20, 1 << 20, 4, 4)):
    import decode_attention_span_gb300 as sk
    from decode_attention_span_gb300.kv4 import SekvKv4Cache
    return (ctypes.byref(sk.Config(*cfg, 0, 0, 64).c()), None if cache is None else ctypes.byref(SekvKv4Cache(*cache)))


def test_tree_and_keep_refusals(libsekv):
    def tree(a=cache_args(), dt=0, q=P, n=3, first=P, t=P, stride=3, scale=1.0, ws=P):
        return libsekv.sekv_kv4_tree_attention(*a, dt, q, n, first, t, stride, scale, P, P, ws, 0, None)

    def keep(a=cache_args(), first=P, k=P, n=3, n_keep=P, ws=P):
        return libsekv.sekv_kv4_keep(*a, first, k, n, n_keep, ws, 0, None)
    for f in (tree, keep):
        assert f(cache_args(cfg=(1025, 8, 2))) == UNSUPPORTED
        assert f(cache_args(cache=None)) == INVALID and f(ws=None) == INVALID and f(first=None) == INVALID
        assert f(cache_args(cache=(1 << 20, 1 << 20, 0, 4))) == INVALID
    for kw in (dict(dt=2), dict(q=None), dict(q=ODD), dict(t=None), dict(t=ctypes.c_void_p((1 << 20) + 4)), dict(stride=-1),
               dict(scale=0.0), dict(scale=math.nan), dict(scale=3e38)):
        assert tree(**kw) == INVALID, kw
    for n in (0, -1, 65):
        assert tree(n=n) == UNSUPPORTED
    assert tree(cache_args(cache=(1 << 20, 1 << 20, 4, 1 << 24))) == UNSUPPORTED
    assert keep(k=None) == INVALID and keep(n=-1) == INVALID and keep(n=65) == UNSUPPORTED
    assert keep(n=0) == 0 and keep(k=None, n=0) == 0


def test_states_refusals(libsekv):
    big = ctypes.c_size_t(1 << 40)

    def call(x=P, dt=0, n=2, d=64, xs=64, w=P, V=9, wst=64, tok=P, wide=0, scale=1.0, lp=P, ws=P, size=big):
        return libsekv.sekv_states_logprobs(x, dt, n, d, xs, w, V, wst, tok, wide, scale, lp, None, 0, ws, size, None)

    def backward(x=P, dt=0, n=2, d=64, xs=64, w=P, V=9, wst=64, tok=P, wide=0, scale=1.0, lse=P, dx=None, dw=None, ws=P, size=big):
        return libsekv.sekv_states_logprobs_backward(x, dt, n, d, xs, w, V, wst, tok, wide, scale, lse, None, None, dx, dw, 0, ws, size, None)
    for f in (call, backward):
        for kw in (dict(x=None), dict(x=ODD), dict(dt=2), dict(n=-1), dict(d=0), dict(d=12), dict(xs=60), dict(xs=56), dict(w=None),
                   dict(w=ODD), dict(V=0), dict(wst=63), dict(wst=32), dict(tok=None), dict(tok=ctypes.c_void_p((1 << 20) + 2)),
                   dict(wide=1, tok=ctypes.c_void_p((1 << 20) + 4)), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
                   dict(scale=3e38), dict(ws=None), dict(ws=ODD)):
            assert f(**kw) == INVALID, kw
        assert f(n=1 << 31) == UNSUPPORTED and f(V=(1 << 30) + 1) == UNSUPPORTED and f(d=1 << 25, xs=1 << 25, wst=1 << 25) == UNSUPPORTED
        assert f(size=ctypes.c_size_t(1000)) == -2
        assert f(n=0) == 0 and f(n=0, x=None, tok=None) == 0
    assert call(lp=None) == INVALID
    assert backward(lse=None) == INVALID and backward(dx=ODD) == INVALID and backward() == 0  # no gradient wanted
    H = lambda B, T, out=P: libsekv.sekv_states_surprisal(P, 0, B, T, 64, 64, P, 9, 64, P, 0, out, 0, P, big, None)  # noqa: E731
    assert H(-1, 2) == INVALID and H(1, -2) == INVALID and H(1, 2, None) == INVALID and H(0, 5) == 0 and H(3, 0) == 0
    assert H(1 << 32, 1) == UNSUPPORTED and H(1 << 16, 1 << 16) == UNSUPPORTED


def test_states_workspace_grows_with_each_size(libsekv):
    """So that the workspace of a large call serves every smaller one."""
    size = libsekv.sekv_states_workspace_size
    rows, vocab, dim = (1, 7, 128, 129, 5000, 8192, 20000, 100000), (1, 224, 225, 257, 9000, 50021, 200000), (8, 200, 4096)
    for back in (0, 1):
        for r in range(len(rows)):
            for v in range(len(vocab)):
                for d in range(len(dim)):
                    n = size(rows[r], vocab[v], dim[d], back)
                    assert n >= 512
                    for r2, v2, d2 in ((max(r - 1, 0), v, d), (r, max(v - 1, 0), d), (r, v, max(d - 1, 0))):
                        assert size(rows[r2], vocab[v2], dim[d2], back) <= n
                    assert size(rows[r], vocab[v], dim[d], 0) <= size(rows[r], vocab[v], dim[d], 1)
    assert size(-1, 9, 8, 0) == 0 and size(1, 0, 8, 0) == 0 and size(1, 9, 0, 1) == 0 and size(1 << 31, 9, 8, 0) == 0


def test_bindings_refuse_tensors_off_the_gpu(libsekv):
    import torch
    import decode_attention_span_gb300 as sk
    x, w, t = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    for f in (lambda: sk.states_logprobs(x, w, t, None), lambda: sk.states_surprisal(x[None], w, t[None], None),
              lambda: sk.states_logprobs_backward(x, w, t, None, None, None)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        sk.states_surprisal(x, w, t, None)
