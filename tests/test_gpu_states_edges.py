"""GPU: log-probabilities from last states and their gradient where it is easy to go wrong: waits that run out,
factors far apart, long sums."""
import time

import pytest
import torch

from test_gpu_states import check_states, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sk():
    from decode_attention_span_gb300 import build
    build.build()
    import decode_attention_span_gb300 as sk
    return sk


@pytest.mark.parametrize("T", [129, 300, 511, 1024])
@pytest.mark.parametrize("D", [64, 520, 4096])
def test_pairs_that_give_up_end_at_once(sk, T, D):
    """With waits that run out at once each CTA of a pair stops copying where it is.  The pair ends when the copies
    that were issued have come, which none of those that were not can hold up (for a limit of 2 s)."""
    V = 3001
    x, w, tok = (t.cuda() for t in inputs("bf16", T, V, D, 6))
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    g = torch.ones(T, device="cuda")
    want = sk.states_logprobs(x, w, tok, ws)
    grads = sk.states_logprobs_backward(x, w, tok, want.lse, g, ws)
    assert ws.status() == (0, 0)
    t0 = time.monotonic()
    for _ in range(5):
        sk.states_logprobs(x, w, tok, ws, flags=2)
        sk.states_logprobs_backward(x, w, tok, want.lse, g, ws, flags=2)
    assert ws.status()[0] == 2
    assert time.monotonic() - t0 < 1.0
    got = sk.states_logprobs(x, w, tok, ws)
    again = sk.states_logprobs_backward(x, w, tok, want.lse, g, ws)
    assert ws.status() == (0, 0) and torch.equal(got.lse, want.lse) and torch.equal(got.logprob, want.logprob)
    assert torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])


def rounding_ratios(sk, dtype, n, scale=1.0):
    """Errors of d_states and d_weight of a mean over n rows (times 1024, away from f16's smallest numbers), in units of
    the error that rounding the exact ones alone has."""
    V, D = 4000, 64
    x, w, tok = inputs(dtype, n, V, D, n)
    ws = sk.StatesWorkspace(n, V, D, backward=True)
    g = torch.full((n,), -1024.0 / n, device="cuda")
    lse = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws, scale=scale).lse
    got = sk.states_logprobs_backward(x.cuda(), w.cuda(), tok.cuda(), lse, g, ws, scale=scale)
    h, m = x.double(), w.double()
    G = torch.softmax(h @ m.T * scale, 1)
    G[torch.arange(n), tok] -= 1
    G *= scale * 1024.0 / n
    return [float((a.cpu().double() - b).norm() / (b.to(x.dtype).double() - b).norm()) for a, b in zip(got, (G @ m, G.T @ h))]


@pytest.mark.parametrize("dtype,n", [("bf16", 1021), ("bf16", 600), ("bf16", 300), ("bf16", 1024), ("fp16", 1000), ("fp16", 200), ("fp16", 1021)])
def test_gradient_of_a_mean_for_any_number_of_rows(sk, dtype, n):
    """G's roundings are independent of each other: their error in the results is at most as large as the results' own
    roundings', in the mean square, so that both together are at most sqrt(2) of those (2% for the sample).  One and
    the same rounding of 1 / n in all rows would be more: 1.5 to 2.1 times at these n, at a power of two."""
    assert max(rounding_ratios(sk, dtype, n)) < 2 ** 0.5 * 1.02


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale,size", [(2.0 ** 100, 2.0 ** -104), (2.0 ** -30, 2.0 ** 34), (2.0 ** 120, 2.0 ** -120)])
def test_gradient_of_scales_and_factors_that_cancel(sk, dtype, scale, size):
    """Factor times scale is of ordinary size, though neither of the two is.  All logits are 0: states and weight
    share no dimension."""
    T, V, D = 40, 300, 64
    h, m, tok = inputs(dtype, T, V, D, 3)
    h[:, 32:], m[:, :32] = 0, 0
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    g = torch.full((T,), size, device="cuda")
    lse = sk.states_logprobs(h.cuda(), m.cuda(), tok.cuda(), ws, scale=scale).lse
    got = sk.states_logprobs_backward(h.cuda(), m.cuda(), tok.cuda(), lse, g, ws, scale=scale)
    assert ws.status() == (0, 0)
    G = torch.full((T, V), -1.0 / V, dtype=torch.float64)
    G[torch.arange(T), tok] += 1
    G *= size * scale
    # each element of G and each result is off by half a step, and the probabilities by 2^-20
    eps = torch.finfo(h.dtype).eps
    for a, want, size in zip(got, (G @ m.double(), G.T @ h.double()), (G.abs() @ m.double().abs(), G.abs().T @ h.double().abs())):
        assert ((a.cpu().double() - want).abs() <= 1.05 * eps * size + (2.0 ** -25 if dtype == "fp16" else 0)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("pad", [1e30, 3e38, float("inf"), float("nan")])
def test_gradient_beside_padding_with_anything_in_it(sk, dtype, ids, pad):
    """The factor on a row without a token counts for nothing, whatever it is: the same bits as with 0 there."""
    T, V, D = 200, 300, 64
    x, w, tok = (t.cuda() for t in inputs(dtype, T, V, D, 5))
    tok = tok.to(ids)
    tok[::3] = -1
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    g = torch.randn(T, generator=torch.Generator().manual_seed(1)).cuda()
    g[::3] = 0
    lse = sk.states_logprobs(x, w, tok, ws).lse
    want = sk.states_logprobs_backward(x, w, tok, lse, g, ws)
    g[::3] = pad
    got = sk.states_logprobs_backward(x, w, tok, lse, g, ws)
    assert ws.status() == (0, 0) and not got[0][::3].any()
    for a, b in zip(got, want):
        assert a.any() and torch.equal(a, b)


def exact_gradient(x, w, tok, g, e):
    """d_states and d_weight in 64 bits, of tensors on the GPU."""
    m = w.double()
    dx, dw = torch.empty(x.shape, dtype=torch.float64, device="cuda"), torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for i in range(0, x.shape[0], 1024):
        h, t, gi = x[i:i + 1024].double(), tok[i:i + 1024], g[i:i + 1024].double()
        gi = torch.where(t >= 0, gi, 0.0)
        G = torch.softmax(h @ m.T, 1) * (e[i:i + 1024].double() - gi)[:, None]
        G[torch.arange(len(t)), t.clamp(min=0)] += gi
        dx[i:i + 1024] = G @ m
        dw += G.T @ h
    return dx, dw


@pytest.mark.parametrize("T,V,D", [(1024, 32000, 4096), (60000, 8000, 512), (9000, 70000, 256)])
def test_long_sums_of_one_sign_are_not_cut_off(sk, T, V, D):
    """Positive factors, states and weights: errors of the sums would all point one way.  4096 of K are 256 additions of 16
    products to a sum that grows evenly, each cut off by at most 17 * 2^-25 of it, and what comes after is rounded; the mean
    error beyond the results' own rounding is at most that, however long the sum."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.rand(n, D, generator=g, device="cuda") * 0.5 + 0.75 for n in (T, V))
    x[:, D // 2:] = 0
    w[:, :D // 2] = 0     # logits from the first dimension alone
    x[:, 0], w[:, 0] = (torch.randn(n, generator=g, device="cuda") for n in (T, V))
    x, w = x.half(), w.half()
    tok, zero, one = torch.full((T,), -1, device="cuda"), torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    lse = sk.states_logprobs(x, w, tok, ws).lse
    got = sk.states_logprobs_backward(x, w, tok, lse, None, ws, grad_lse=one)
    assert ws.status() == (0, 0)
    for a, want, at in zip(got, exact_gradient(x, w, tok, zero, one), (slice(D // 2, D), slice(1, D // 2))):
        a, want = a.double()[:, at], want[:, at]
        bias = ((a - want.half().double()) / want).mean().item()
        assert abs(bias) <= 17 * 2.0 ** -25 * 128 + 2.0 ** -18, bias


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gradient_of_pieces_whose_last_tiles_are_cut(sk, dtype):
    """10000 rows take 13312 tokens at a time, and 4 of the 80 tiles of d_states have their sums cut into shares in each
    piece: those of earlier pieces join them.  Each tile on its own, against 64 bits: G and the result are rounded by half
    a step each."""
    T, V, D = 10000, 30000, 512
    x, w, tok = (t.cuda() for t in inputs(dtype, T, V, D, 6))
    tok[::11] = -1
    ws = sk.StatesWorkspace(T, V, D, backward=True)
    g, e = (torch.randn(T, generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2))
    lse = sk.states_logprobs(x, w, tok, ws).lse
    dx, dw = sk.states_logprobs_backward(x, w, tok, lse, g, ws, grad_lse=e)
    assert ws.status() == (0, 0)
    half = torch.finfo(x.dtype).eps / 2
    for a, want in zip((dx, dw), exact_gradient(x, w, tok, g, e)):
        for i in range(0, want.shape[0], 256):
            for j in range(0, D, 256):
                u, v = a[i:i + 256, j:j + 256].double(), want[i:i + 256, j:j + 256]
                assert float((u - v).norm() / v.norm()) <= 2 * half, (i, j)
    # one without the other
    only, _ = sk.states_logprobs_backward(x, w, tok, lse, g, ws, grad_lse=e, want_weight=False)
    assert torch.equal(only, dx)


@pytest.mark.parametrize("T", [8192, 8193, 8200, 8320, 16390])
def test_rows_behind_the_last_whole_part(sk, T):
    """Rows are taken 8192 at a time; a few that are left go through the kernel of one CTA, with tiles of its own width."""
    V, D = 1100, 72
    x, w, tok = inputs("bf16", T, V, D, 4)
    ws = sk.StatesWorkspace(T, V, D)
    r = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), ws)
    at = [0, 1, 4096, 8190, 8191] + list(range(8192, T, 97)) + [T - 1]
    check_states(sk.StatesLogprobs(r.logprob[at], r.lse[at]), x[at], w, tok[at])
    assert ws.status() == (0, 0)
