"""GPU parity of the log-probabilities from last states, the surprisal and the gradient against their fp64
oracles."""
import math

import numpy as np
import pytest
import torch

from oracle import tokens
from test_gpu_operators import DT, HALF, INF, compare, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sk():
    from decode_attention_span_gb300 import build
    build.build()
    import decode_attention_span_gb300 as sk
    return sk


def inputs(dtype, T, V, D, seed=0, spread=2.5):
    x = torch.randn(T, D, generator=gen(seed))
    w = torch.randn(V, D, generator=gen(seed + 1)) * (spread / math.sqrt(D))
    tok = torch.randint(0, V, (T,), generator=gen(seed + 2))
    return x.to(DT[dtype]), w.to(DT[dtype]), tok


def product_error(x, w, scale):
    """Of a logit: each instruction adds 16 products to its sum, all cut off 25 bits under the largest,
    which is 17 * 2^-25 of the sum of the products' sizes at most; 64 of them make a sum, and those are
    added with roundings of 2^-24."""
    size = abs(scale) * (np.abs(x) @ np.abs(w).T)
    steps = min(64, -(-x.shape[1] // 16))
    return size * (steps * 17 * 2.0 ** -25 + (x.shape[1] / 1024 + 2) * 2.0 ** -24)


def check_states(r, x, w, tok, scale=1.0):
    x, w = x.double().numpy(), w.double().numpy()
    ref = tokens.states_logprobs(x, w, tok.numpy().reshape(-1), scale)
    d = product_error(x, w, scale).max(1)
    # the exponent's fma errs by 2^-23 of the logit to the base 2, the exponential by 2^-22, sums of 128
    # numbers and of the tiles by 2^-24 a step
    big = np.abs(x @ w.T * scale).max(1)
    d = d + 2.0 ** -22 * big + 2.0 ** -22 + 2.0 ** -24 * (w.shape[0] / 128 / 32 + 80)
    for name in ("logprob", "lse"):
        want = ref[name]
        compare(getattr(r, name).double().cpu().numpy().reshape(-1), want, 2 * d + 2.0 ** -22 * np.abs(np.where(np.isfinite(want), want, 0)), name)


CASES = [(1, 1, 8), (1, 300, 8), (3, 7, 16), (2, 257, 72), (17, 1000, 200), (127, 999, 64), (128, 2048, 128), (129, 1025, 136),
         (255, 256, 1032), (256, 255, 1024), (257, 513, 2056), (300, 5000, 520), (1000, 1, 64), (9000, 130, 24)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,V,D", CASES)
def test_states_logprobs(sk, dtype, T, V, D):
    x, w, tok = inputs(dtype, T, V, D, T)
    tok[::5] = -1
    ws = sk.StatesWorkspace(T, V, D)
    r = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws, scale=0.75)
    assert ws.status() == (0, 0)
    check_states(r, x, w, tok, 0.75)
    r2 = sk.states_logprobs(x.cuda(), w.cuda(), tok.int().cuda(), sk.StatesWorkspace(2 * T, V + 500, D + 8, backward=True), scale=0.75)
    assert torch.equal(r.logprob, r2.logprob) and torch.equal(r.lse, r2.lse)


def test_states_strides(sk):
    """Rows and vocabulary rows further apart than they are long, and sequences side by side."""
    x, w, tok = inputs("bf16", 60, 300, 40, 5)
    ws = sk.StatesWorkspace(60, 300, 40)
    want = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws)
    wide_x, wide_w = torch.full((60, 96), math.nan).bfloat16().cuda(), torch.full((300, 64), math.nan).bfloat16().cuda()
    wide_x[:, 8:48], wide_w[:, 16:56] = x.cuda(), w.cuda()
    got = sk.states_logprobs(wide_x[:, 8:48], wide_w[:, 16:56], tok.cuda(), ws)
    assert torch.equal(got.logprob, want.logprob) and torch.equal(got.lse, want.lse)
    got = sk.states_logprobs(wide_x[:, 8:48].view(4, 15, 40), wide_w[:, 16:56], tok.cuda().view(4, 15), ws)
    assert got.lse.shape == (4, 15) and torch.equal(got.lse.view(-1), want.lse)
    one = sk.states_logprobs(wide_x[7:8, 8:48], wide_w[:, 16:56], tok[7:8].cuda(), ws)
    assert torch.equal(one.lse, want.lse[7:8])
    # every second position of two sequences; rows that are not evenly spaced are refused
    got = sk.states_logprobs(x.cuda()[::2].view(2, 15, 40), w.cuda(), tok.cuda()[::2].contiguous().view(2, 15), ws)
    assert torch.equal(got.lse.view(-1), want.lse[::2])
    with pytest.raises(ValueError):
        sk.states_logprobs(x.cuda().view(4, 15, 40)[:, :7], w.cuda(), tok.cuda().view(4, 15)[:, :7].contiguous(), ws)


def test_states_refusals_of_the_binding(sk):
    x, w, tok = (t.cuda() for t in inputs("bf16", 4, 30, 16))
    ws = sk.StatesWorkspace(4, 30, 16)
    for bad in (lambda: sk.states_logprobs(x, w, tok, sk.Workspace(sk.Config(1, 1, 1, 0, 0, 64))),
                lambda: sk.states_logprobs(x, w[:, :8], tok, ws), lambda: sk.states_logprobs(x, w.T.contiguous().T, tok, ws),
                lambda: sk.states_logprobs(x, w, tok[:3], ws), lambda: sk.states_logprobs(x, w, tok.repeat(2)[::2], ws),
                lambda: sk.states_surprisal(x, w, tok, ws),
                lambda: sk.states_logprobs_backward(x, w, tok, tok.float()[:3], None, ws),
                lambda: sk.states_logprobs_backward(x, w, tok, tok.float(), None, ws, d_weight=torch.empty(30, 8).bfloat16().cuda())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sk.states_logprobs(x.float(), w.float(), tok, ws), lambda: sk.states_logprobs(x, w.half(), tok, ws),
                lambda: sk.states_logprobs(x, w, tok.float(), ws), lambda: sk.states_logprobs_backward(x, w, tok, tok, None, ws)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(sk.SekvError):
        sk.states_logprobs(x[:, :12], w[:, :12], tok, ws)       # 12 dimensions
    many = torch.zeros(400, 16, dtype=torch.bfloat16, device="cuda"), w, torch.zeros(400, dtype=torch.int64, device="cuda")
    with pytest.raises(sk.SekvError):  # parts are rounded up to 256 bytes: a few rows more may still fit
        sk.states_logprobs(*many, ws)
    with pytest.raises(sk.SekvError):
        sk.states_logprobs_backward(x, w, tok, tok.float(), None, ws)  # made without backward


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [5, 200])
def test_states_special_rows(sk, dtype, T):
    """NaN and infinite states, logits of -inf, tokens that are none: a row's own affair."""
    V, D = 700, 64
    x, w, tok = inputs(dtype, T, V, D, 3)
    x[:, 0], w[:, 0] = 1.0, 0.0
    w[5, 0] = -INF            # a masked token: logit -inf in every row
    x[1, 3], x[2, 7] = math.nan, INF
    tok[0], tok[3], tok[4] = 5, V, -2
    w[:, 7] = w[:, 7].abs()   # +inf logits in row 2
    ws = sk.StatesWorkspace(T, V, D)
    r = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws)
    assert ws.status() in ((1, 3), (1, 4))
    assert r.logprob[0].item() == -INF and math.isfinite(r.lse[0])
    for i in (1, 2):
        assert math.isnan(r.logprob[i]) and math.isnan(r.lse[i])
    for i in (3, 4):
        assert math.isnan(r.logprob[i]) and math.isfinite(r.lse[i])
    keep = [i for i in range(T) if i not in (1, 2, 3, 4)]
    y = x.double().numpy()[keep] @ np.where(np.isinf(w.double().numpy()), 0, w.double().numpy()).T
    y[:, 5] = -INF
    ref = tokens.token_logprobs(y, tok.numpy()[keep])
    d = product_error(x.double().numpy()[keep], np.where(np.isinf(w.double().numpy()), 0, w.double().numpy()), 1.0).max() + 1e-5
    for name in ("logprob", "lse"):
        compare(getattr(r, name).double().cpu().numpy()[keep], ref[name], 2 * d, name)
    # nothing but -inf
    r = sk.states_logprobs(x[:1].cuda(), w[5:6].cuda(), torch.tensor([0]).cuda(), ws)
    assert r.lse.item() == -INF and r.logprob.item() == -INF
    r = sk.states_logprobs(x[:1].cuda(), w[5:6].cuda(), torch.tensor([-1]).cuda(), ws)
    assert r.lse.item() == -INF and r.logprob.item() == 0


def test_states_logits_far_apart(sk):
    """One row's likeliest token outweighs all, another's are all alike, and logits in the thousands."""
    x, w, tok = inputs("bf16", 3, 1200, 64, 8)
    x[1] = 0
    x[2] *= 400
    ws = sk.StatesWorkspace(3, 1200, 64)
    r = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws)
    check_states(r, x, w, tok)
    assert abs(r.lse[1].item() - math.log(1200)) < 1e-5


@pytest.mark.parametrize("B,T,V,D", [(1, 1, 50, 8), (3, 2, 60, 16), (2, 100, 700, 64), (4, 333, 260, 72), (1, 9001, 33, 8)])
def test_states_surprisal(sk, B, T, V, D):
    x, w, tok = inputs("bf16", B * T, V, D, 4)
    tok[::7] = -1
    x, tok = x.view(B, T, D), tok.view(B, T)
    ws = sk.StatesWorkspace(B * T, V, D)
    H = sk.states_surprisal(x.cuda(), w.cuda(), tok.cuda(), ws)
    assert ws.status() == (0, 0) and not H[:, 0].any()
    # the same as the log-probabilities of the tokens that follow
    nxt = torch.cat([tok[:, 1:], torch.full((B, 1), -1)], 1).contiguous()
    lp = sk.states_logprobs(x.cuda(), w.cuda(), nxt.cuda(), ws).logprob
    assert torch.equal(H[:, 1:], 0.0 - lp[:, :-1])
    out = torch.full((B, T), 7.0, device="cuda")
    assert sk.states_surprisal(x.cuda(), w.cuda(), tok.int().cuda(), ws, out=out) is out and torch.equal(out, H)
    if B * T < 2000:
        ref = tokens.surprisal((x.double().numpy() @ w.double().numpy().T), tok.numpy())
        d = product_error(x.double().numpy().reshape(B * T, D), w.double().numpy(), 1.0).max() + 2e-5
        compare(H.double().cpu().numpy(), ref, 2 * d, "H")


# ------------------------------------------------------------------ the gradient
def check_gradient(dx, dw, x, w, tok, g, e, scale, dtype):
    """An element of G is rounded by half a step (f16: of no less than 2^-38 of the largest factor on a row) and
    errs by what its exponent does; the sums by 17 * 2^-25 of their terms' sizes an instruction and 2^-24 a
    piece; the result is rounded by half a step."""
    x, w, tok = x.double().numpy(), w.double().numpy(), tok.numpy()
    rdx, rdw, G = tokens.states_gradient(x, w, tok, g, e, scale)
    on = np.where(tok >= 0, g, 0.0)
    factor = scale * (np.abs(e - on) + np.abs(on))
    d = product_error(x, w, scale).max(1) + 2.0 ** -20 + 2.0 ** -21 * np.abs(x @ w.T * scale).max(1)
    y = x @ w.T * scale
    p = np.exp(y - y.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    err = HALF[dtype] * np.abs(G) + 2 * d[:, None] * p * (scale * np.abs(e - on))[:, None] + 2.0 ** -23 * factor[:, None] * p
    if dtype == "fp16":
        err = err + 2.0 ** -38 * factor.max()
    T, V = G.shape
    for got, want, er, size, n in ((dx, rdx, err @ np.abs(w), np.abs(G) @ np.abs(w), V), (dw, rdw, err.T @ np.abs(x), np.abs(G).T @ np.abs(x), T)):
        tol = er + size * (-(-n // 16) * 17 * 2.0 ** -25 + 2.0 ** -20)
        tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "fp16" else 1e-38)
        compare(got.double().cpu().numpy().reshape(want.shape), want, tol, "gradient")
        rel = np.linalg.norm(got.double().cpu().numpy().reshape(want.shape) - want) / max(np.linalg.norm(want), 1e-300)
        assert rel <= 2 * HALF[dtype] or np.linalg.norm(want) < 1e-5, rel  # two roundings, each below half a step


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,V,D", [(1, 40, 8), (3, 300, 72), (96, 1500, 264), (130, 700, 520), (500, 999, 128), (257, 257, 1000),
                                   (2000, 33, 48)])
def test_states_gradient(sk, dtype, T, V, D):
    x, w, tok = inputs(dtype, T, V, D, T + 1)
    tok[1::6] = -1
    rng = np.random.default_rng(T)
    g, e = rng.normal(size=T).astype(np.float32), rng.normal(size=T).astype(np.float32)
    g[2::9] = e[2::9] = 0
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    c = (x.cuda(), w.cuda(), tok.cuda())
    lse = sk.states_logprobs(*c, ws, scale=0.6).lse
    gc, ec = torch.from_numpy(g).cuda(), torch.from_numpy(e).cuda()
    dx, dw = sk.states_logprobs_backward(*c, lse, gc, ws, grad_lse=ec, scale=0.6)
    assert ws.status() == (0, 0) and dx.dtype == x.dtype and dw.shape == w.shape
    check_gradient(dx, dw, x, w, tok, g.astype(float), e.astype(float), 0.6, dtype)
    # rows whose factors are 0
    assert not dx[torch.from_numpy((e == 0) & ((g == 0) | (tok.numpy() < 0))).cuda()].any()
    # each alone, into given tensors, with one of the gradients
    only, none = sk.states_logprobs_backward(*c, lse, gc, ws, grad_lse=ec, scale=0.6, want_weight=False)
    assert none is None and torch.equal(only, dx)
    out = torch.full_like(dw, 9.0)
    none, only = sk.states_logprobs_backward(*c, lse, gc, ws, grad_lse=ec, scale=0.6, want_states=False, d_weight=out)
    assert none is None and only is out and torch.equal(out, dw)
    dx, dw = sk.states_logprobs_backward(*c, lse, gc, ws, scale=0.6)
    check_gradient(dx, dw, x, w, tok, g.astype(float), 0 * e.astype(float), 0.6, dtype)
    dx, dw = sk.states_logprobs_backward(*c, lse, None, ws, grad_lse=ec, scale=0.6)
    check_gradient(dx, dw, x, w, tok, 0 * g.astype(float), e.astype(float), 0.6, dtype)


@pytest.mark.parametrize("size", [1e-30, 1e-7, 1e4])
def test_states_gradient_of_small_and_large_factors(sk, size):
    """Factors on the loss far from 1: f16's G follows the largest."""
    x, w, tok = inputs("fp16", 40, 500, 64, 2)
    g = np.full(40, size, np.float32)
    ws = sk.StatesWorkspace(40, 500, 64, backward=True)
    lse = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws).lse
    dx, dw = sk.states_logprobs_backward(x.cuda(), w.cuda(), tok.cuda(), lse, torch.from_numpy(g).cuda(), ws)
    check_gradient(dx, dw, x, w, tok, g.astype(float), np.zeros(40), 1.0, "fp16")


def test_states_gradient_in_pieces_of_the_vocabulary(sk):
    """More than one piece: 17000 rows take 8192 tokens at a time; against the products of the pieces' parts."""
    T, V, D = 17000, 20000, 64
    x, w, tok = (t.cuda() for t in inputs("bf16", T, V, D, 6))
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    g = torch.randn(T, generator=gen(1)).cuda()
    lse = sk.states_logprobs(x, w, tok, ws).lse
    dx, dw = sk.states_logprobs_backward(x, w, tok, lse, g, ws)
    want_x, want_w = torch.zeros(T, D, dtype=torch.float64, device="cuda"), torch.zeros(V, D, dtype=torch.float64, device="cuda")
    for i in range(0, T, 2000):
        h, t = x[i:i + 2000].double(), tok[i:i + 2000]
        G = -torch.softmax(h @ w.double().T, 1)
        G[torch.arange(len(t)), t] += 1
        G *= g[i:i + 2000, None].double()
        want_x[i:i + 2000] = G @ w.double()
        want_w += G.T @ h
    for got, want in ((dx, want_x), (dw, want_w)):
        assert float((got.double() - want).norm() / want.norm()) <= 2 * HALF["bf16"]
    none, again = sk.states_logprobs_backward(x, w, tok, lse, g, ws, want_states=False)
    assert torch.equal(again, dw)


def test_states_gradient_against_differences(sk):
    """Of the call's own loss, along random directions, in f16 with a step that its states can take."""
    T, V, D = 24, 300, 64
    x, w, tok = inputs("fp16", T, V, D, 9)
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    g = torch.randn(T, generator=gen(4)).cuda()
    r = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws)
    dx, dw = sk.states_logprobs_backward(x.cuda(), w.cuda(), tok.cuda(), r.lse, g, ws)
    for seed in range(4):
        step = (torch.randint(0, 3, (T, D), generator=gen(seed)) - 1).float() * 2.0 ** -6
        up, down = (x.float() + step).half(), (x.float() - step).half()
        a, b = (sk.states_logprobs(y.cuda(), w.cuda(), tok.cuda(), ws).logprob for y in (up, down))
        diff = float(((a - b).double() * g.double()).sum())
        want = float((dx.double().cpu() * (up.double() - down.double())).sum())
        # third order: |step . w|^3 of some (2^-6 sqrt(D) 2.5 / sqrt(D) * 3)^3 a row, and f16's half steps
        bound = T * 2 * (2.0 ** -6 * 7.5) ** 3 + float((dx.double().cpu().abs() * (up.double() - down.double()).abs()).sum()) * 2.0 ** -10
        assert abs(diff - want) <= bound, (diff, want, bound)


def test_states_of_nothing(sk):
    w = torch.randn(50, 16, generator=gen(1)).bfloat16().cuda()
    ws = sk.StatesWorkspace(4, 50, 16, backward=True)
    x, tok = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    r = sk.states_logprobs(x, w, tok, ws)
    assert r.lse.shape == (0,)
    dw = torch.full_like(w, 3.0)
    dx, got = sk.states_logprobs_backward(x, w, tok, r.lse, None, ws, d_weight=dw)
    assert dx.shape == (0, 16) and got is dw and not dw.any()
    assert sk.states_surprisal(x.view(0, 5, 16), w, tok.view(0, 5), ws).shape == (0, 5)
    assert ws.status() == (0, 0)


def test_states_short_waits_time_out_and_leave_the_gpu_usable(sk):
    for T in (3, 500):
        x, w, tok = (t.cuda() for t in inputs("bf16", T, 3000, 512, 6))
        ws = sk.StatesWorkspace(T, 3000, 512, backward=True)
        g = torch.ones(T, device="cuda")
        want = sk.states_logprobs(x, w, tok, ws)
        grads = sk.states_logprobs_backward(x, w, tok, want.lse, g, ws)
        sk.states_logprobs(x, w, tok, ws, flags=2)
        assert ws.status()[0] == 2
        sk.states_logprobs_backward(x, w, tok, want.lse, g, ws, flags=2)
        assert ws.status()[0] == 2
        got = sk.states_logprobs(x, w, tok, ws)
        again = sk.states_logprobs_backward(x, w, tok, want.lse, g, ws)
        assert ws.status() == (0, 0) and torch.equal(got.lse, want.lse) and torch.equal(got.logprob, want.logprob)
        assert torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])


def test_states_on_a_side_stream_and_in_a_graph(sk):
    """Loss and gradient eagerly on another stream, and captured, replayed with other inputs."""
    T, V, D = 300, 3000, 256
    x, w, tok = (t.cuda() for t in inputs("bf16", T, V, D, 6))
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    g = torch.full((T,), -1.0 / T, device="cuda")

    def step(stream=None):
        r = sk.states_logprobs(x, w, tok, ws, stream=stream)
        return [*r, *sk.states_logprobs_backward(x, w, tok, r.lse, g, ws, stream=stream)]
    want = [y.clone() for y in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for again in range(2):
        if again:
            x.neg_()
            w.mul_(2)
        graph.replay()
        got = [y.clone() for y in held]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert ws.status() == (0, 0)


def test_a_prefill_scored_from_its_states_marks_the_same_spans(sk):
    """The surprisal from states is that from the logits, and the span build takes it."""
    B, T, V, D = 1, 600, 1000, 128
    x, w, tok = (t.cuda() for t in inputs("bf16", B * T, V, D, 6, spread=4.0))
    x, tok = x.view(B, T, D), tok.view(B, T)
    H = sk.states_surprisal(x, w, tok, sk.StatesWorkspace(B * T, V, D))
    from_logits = sk.surprisal(x.float() @ w.float().T, tok, sk.Workspace(sk.Config(1, 1, 1, 0, 0, 64)))
    assert torch.allclose(H, from_logits, atol=1e-4)
    cfg = sk.Config(B, 4, 1, 4, 16, 256, 16, 4, 64, 4.0)
    K, Vv = (torch.randn(B, 1, T, 128, generator=gen(i)).bfloat16().cuda() for i in (1, 2))
    W = (torch.randn(1, 64, 128, generator=gen(3)) / 11).cuda()
    gates = torch.ones(B, 1, 2, 256, 16, device="cuda")
    out = sk.alloc_cache(cfg, 64 << 20)
    wsb = sk.Workspace(cfg, which=3, ctx_len=T)
    sk.build_spans(cfg, K, Vv, H, W, gates, out, wsb)
    assert wsb.status() == (0, 0) and int(out["n_spans"][0]) > 4
