"""GPU parity of the operators around the cache at the places where they can go wrong, against
their fp64 oracles or closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import tokens

from cases import SCALE, TOL_ABS, decode_case

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
INF = math.inf


@pytest.fixture(scope="module")
def sk():
    from decode_attention_span_gb300 import build
    build.build()
    import decode_attention_span_gb300 as sk
    return sk


@pytest.fixture(scope="module")
def ws(sk):
    return sk.Workspace(sk.Config(1, 1, 1, 0, 0, 64))


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ log-probabilities
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,top", [(200, 32), (500, 20), (2000, 32)])
def test_alternatives_of_short_rows_with_masked_first_ids(sk, ws, dtype, vocab, top):
    """Short rows with many alternatives have more candidates than places as a rule and go to the
    exact bound; with the first ids masked the first thread has no element of its own there."""
    x = (torch.randn(700, vocab, generator=gen(vocab)) * 3).to(DT[dtype])
    x[:, :16] = -INF
    x[::3, 16:100] = -INF
    tok = torch.randint(100, vocab, (700,), generator=gen(1))
    want = tokens.token_logprobs(x.double().numpy(), tok.numpy(), 1.0, top)
    xc, tc = x.cuda(), tok.cuda()
    for _ in range(3):
        r = sk.token_logprobs(xc, tc, ws, n_top=top)
        assert np.array_equal(r.top_ids.cpu().numpy(), want["top_ids"])
        # an exponent of up to 40, sums of up to 2000 / 128 + 40 additions, the result's own size
        err = np.abs(r.logprob.double().cpu().numpy() - want["logprob"])
        assert (err <= 3 * (120 * 2.0 ** -24 + 2.0 ** -22 + 56 * 2.0 ** -24) + 2.0 ** -22 * 60).all()
    assert ws.status() == (0, 0)


# ------------------------------------------------------------------ outputs and streams
def small_cache(sk, B, Hkv, hq, T, seed=0, n_q=1):
    """A 4-bit cache that holds T random tokens of each sequence."""
    cfg = sk.Config(B, hq, Hkv, 0, 0, 64)
    mp = -(-T // 64)
    cache = sk.Kv4Cache(cfg, sk.alloc_kv4_pages(cfg, B * mp),
                        torch.arange(B * mp, dtype=torch.int32, device="cuda").view(B, mp))
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q)
    k, v = (torch.randn(B, T, Hkv, 128, generator=gen(seed + i)).bfloat16().cuda() for i in range(2))
    sk.kv4_append(cfg, cache, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"), kws)
    return cfg, cache, kws


def test_outputs_made_for_another_stream(sk, ws):
    """Outputs of a call with stream= are neither filled on the current stream nor taken from its
    freed memory: here the current stream is busy, and has writes to such memory ahead of it."""
    B, T = 2, 40
    cfg, cache, kws = small_cache(sk, B, 2, 4, T)
    i32 = dict(dtype=torch.int32, device="cuda")
    zero, n = torch.zeros(B, **i32), torch.full((B,), 30, **i32)
    q = torch.randn(B, 1, 4, 128, generator=gen(3)).bfloat16().cuda()
    logits, tok = torch.randn(B, T, 300, generator=gen(4)).cuda(), torch.zeros(B, T, dtype=torch.int64, device="cuda")
    plan, pos = sk.RopePlan(128), torch.arange(T, **i32)
    x = torch.randn(B, T, 3, 128, generator=gen(5)).cuda()
    side = torch.cuda.Stream()
    calls = [lambda s: sk.kv4_read(cfg, cache, zero, T, kws, n_valid=n, stream=s),
             lambda s: sk.kv4_read(cfg, cache, zero, T, kws, stream=s),
             lambda s: sk.kv4_attention(cfg, cache, q, n, 0.1, kws, stream=s),
             lambda s: sk.token_logprobs(logits, tok, ws, n_top=3, stream=s),
             lambda s: [sk.surprisal(logits, tok, ws, stream=s)],
             lambda s: sk.rope(plan, x, x[:, :, :1], pos, stream=s)]
    for call in calls:
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        old = [torch.empty_like(t) for t in want for _ in range(2)]
        torch.cuda._sleep(50_000_000)  # some 25 ms
        for t in old:
            t.fill_(7)
        del old, t
        got = call(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_outputs_of_the_span_cache_calls_made_for_another_stream(sk):
    """The same of the calls over the span cache, whose lists and logits start at zero."""
    case = decode_case("llama3_8b_32k", ctx=4096, run_oracle=False)
    w = case.wcfg
    cfg = sk.Config(w.batch, w.n_q_heads, w.n_kv_heads, w.n_sink, w.n_recent, case.tensors["max_spans"],
                    w.rank_cap, w.len_min, w.len_max, w.tau)
    cache = sk.LayerCache({k: v.cuda() for k, v in case.tensors.items() if isinstance(v, torch.Tensor)})
    wsd, side = sk.Workspace(cfg), torch.cuda.Stream()
    q, W, theta = case.q.cuda(), case.W.cuda(), torch.from_numpy(case.theta).cuda()
    q2 = q[:, None].repeat(1, 2, 1, 1)
    lst, cnt, _ = sk.route(cfg, cache, q, W, theta, wsd)
    # no outputs that the kernels leave unwritten: `expanded` of route holds counts entries only
    calls = [lambda s: sk.route(cfg, cache, q, W, theta, wsd, want_z=True, stream=s)[1:],
             lambda s: sk.decode_attention(cfg, cache, q, lst, cnt, SCALE, wsd, stream=s),
             lambda s: sk.decode_step(cfg, cache, q, W, theta, SCALE, wsd, want_list=True, stream=s),
             lambda s: sk.decode_step_noalloc(cfg, cache, q, W, theta, SCALE, want_list=True, stream=s),
             lambda s: sk.decode_step_multi(cfg, cache, q2, W, theta, SCALE, wsd, want_list=True, stream=s)]
    for call in calls:
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        old = [torch.empty_like(t) for t in want for _ in range(2)]
        torch.cuda._sleep(50_000_000)
        for t in old:
            t.fill_(7)
        del old, t
        got = call(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            # the decode kernel's CTAs share the work in the order they come: each result is within
            # TOL_ABS of the exact one, so two are within twice that (a lost one is off by far more)
            assert torch.equal(a, b) if a.dtype == torch.int32 else (a - b).abs().max().item() <= 2 * TOL_ABS
    assert wsd.status() == (0, 0)


@pytest.mark.parametrize("in_place", [False, True])
def test_rotation_directly_before_the_attention(sk, in_place):
    """The attention's blocks may be resident while the rotation still writes their queries; step
    after step the same buffers hold other queries, with nothing launched in between."""
    B, T, hq, n_q = 3, 300, 8, 4
    cfg, cache, kws = small_cache(sk, B, 2, hq, T, n_q=n_q)
    plan = sk.RopePlan(128)
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    x = [torch.randn(B, n_q, hq, 128, generator=gen(i)).bfloat16().cuda() for i in range(30)]
    pos = [torch.full((n_q,), 10 * i, dtype=torch.int32, device="cuda") for i in range(30)]
    want = []
    for q, p in zip(x, pos):
        q = sk.rope(plan, q, None, p)[0]
        torch.cuda.synchronize()
        want.append(sk.kv4_attention(cfg, cache, q, lens, 0.1, kws))
        torch.cuda.synchronize()
    buf = torch.empty_like(x[0])
    src = [q.clone() for q in x]
    got = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    for q, p, (o, l) in zip(src, pos, got):
        r = q if in_place else buf
        sk.rope(plan, q, None, p, q_out=r)
        sk.kv4_attention(cfg, cache, r, lens, 0.1, kws, out=o, lse=l)
    for (o, l), (ow, lw) in zip(got, want):
        assert torch.equal(o, ow) and torch.equal(l, lw)
    assert kws.status() == (0, 0)
