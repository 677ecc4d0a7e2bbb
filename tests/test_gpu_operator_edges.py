"""GPU parity of the operators around the cache at the places where they can go wrong, against
their fp64 oracles or closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import kv4, tokens
from turns import turns

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


@pytest.mark.parametrize("scale", [0.25, 2e-38])
def test_logits_further_apart_than_fp32_reaches(sk, ws, scale):
    """Differences of f32 logits of both signs next to the type's ends are past fp32 before the scale
    brings them back."""
    V = 3000
    x = (torch.rand(6, V, generator=gen(2)) * 2 - 1) * 3.3e38
    x[0, :] = -3.4e38
    x[0, 5] = 3.4e38
    x[1, 2999] = 3.4e38
    x[2, ::2] = torch.randn(V // 2, generator=gen(3))
    tok = torch.tensor([5, 0, 1, 7, 8, 9])
    tok[0] = 17
    r = sk.token_logprobs(x.cuda(), tok.cuda(), ws, n_top=4, scale=scale)
    want = tokens.token_logprobs(x.double().numpy(), tok.numpy(), float(np.float32(scale)), 4)
    assert np.array_equal(r.top_ids.cpu().numpy(), want["top_ids"])
    # three roundings of what an exponent comes from (those below -100 do not count), 2^-22 of the
    # exponential, the sums; a value past fp32 would be an infinity of its sign
    d = 300 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -24 * (V / 128 + 40)
    for name in ("logprob", "top_logprobs", "lse", "entropy"):
        w = want[name]
        g = getattr(r, name).double().cpu().numpy()
        big = np.abs(w) > 3.4e38
        assert np.array_equal(g[big], np.sign(w[big]) * INF), name
        err = np.abs(g - w)[~big]
        assert (err <= 3 * d * (1 + (name == "entropy") * np.abs(w[~big])) + 2.0 ** -22 * np.abs(w[~big])).all(), (name, err.max())


def test_one_likely_token_among_450_million_masked_ones(sk, ws):
    """So many logits at the type's lowest value that their number times their distance, in which
    the entropy's sum is rescaled, comes near fp32's end; all of the weight is on the last."""
    V = 450_000_000
    x = torch.full((1, V), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device="cuda")
    x[0, -1] = 1.0
    r = sk.token_logprobs(x, torch.tensor([V - 1], device="cuda"), ws, n_top=1)
    assert (r.logprob.item(), r.lse.item(), r.entropy.item()) == (0.0, 1.0, 0.0)
    assert (r.top_ids.item(), r.top_logprobs.item()) == (V - 1, 0.0)


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


def test_rotation_in_place_of_a_single_sequence(sk):
    """The same rows seen through another view, whose stride of the single sequence is another:
    still in place."""
    plan, pos = sk.RopePlan(128), torch.arange(5, dtype=torch.int32, device="cuda")
    big = torch.randn(3, 5, 4, 128, generator=gen(1)).bfloat16().cuda()
    want = sk.rope(plan, big[1:2].clone(), None, pos)[0]
    x, y = big[1:2], big[1].unsqueeze(0).as_strided((1, 5, 4, 128), (8, 512, 128, 1), 5 * 4 * 128)
    assert x.data_ptr() == y.data_ptr() and x.stride(0) != y.stride(0)
    sk.rope(plan, x, None, pos, q_out=y)
    assert torch.equal(x, want)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_at_far_positions_by_fifty_digits(sk, inter):
    """Positions up to 2^40 against angles that do not come from the table."""
    pos = [1, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, 12345678901, (1 << 40) - 7]
    plan, w = sk.RopePlan(128, 500000.0, inter), turns(128, 500000.0)
    x = torch.randn(1, len(pos), 2, 128, generator=gen(3)).cuda()
    got = sk.rope(plan, x, None, torch.tensor([pos], device="cuda"))[0].double().cpu().numpy()
    for t, p in enumerate(pos):
        angle = np.array([float(p * v % 1) * 2 * math.pi for v in w])
        want = tokens.rope(x[:, t:t + 1].double().cpu().numpy(), [[1]], angle, 1.0, inter)
        # the table's error, and fp32's: the fraction of a half turn, the sine, three operations
        assert np.abs(got[:, t:t + 1] - want).max() <= 2 * 5 * (p * 2.0 ** -49 + 2.0 ** -22), p


def test_calls_on_nothing(sk, ws):
    """No tokens, no sequences, no heads: empty outputs, nothing written, nothing flagged."""
    cfg, cache, kws = small_cache(sk, 2, 2, 4, 70)
    pages = cache.pages.clone()
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    k = torch.empty(2, 0, 2, 128, dtype=torch.bfloat16, device="cuda")
    sk.kv4_append(cfg, cache, k, k, zero, kws)
    r = sk.kv4_read(cfg, cache, zero, 0, kws, n_valid=zero)
    assert r[0].shape == (2, 2, 0, 128) and torch.equal(cache.pages, pages)
    plan = sk.RopePlan(128)
    for B, T, h in ((2, 0, 3), (0, 4, 3), (2, 4, 0)):
        x = torch.empty(B, T, h, 128, device="cuda")
        q, kk = sk.rope(plan, x, x, torch.zeros(B, T, dtype=torch.int64, device="cuda"))
        assert q.shape == kk.shape == x.shape
    for B, T in ((0, 3), (2, 0)):
        t = torch.zeros(B, T, dtype=torch.int64, device="cuda")
        x = torch.empty(B, T, 50, device="cuda")
        assert sk.token_logprobs(x, t, ws, n_top=2).top_ids.shape == (B, T, 2)
        assert sk.surprisal(x, t, ws).shape == (B, T)
    assert kws.status() == (0, 0) and ws.status() == (0, 0)


# ------------------------------------------------------------------ the 4-bit attention's precision
# What a call may be off by, of the softmax-weighted mean of |z| + 15 |s| (per group of dimensions;
# `bound` of the oracle):
#   2^-22   a weight p s as two f16 numbers, each rounded by half a step, 2^-11 of 2^-11 of it, and
#           2^-25 of the largest weight with it where that is more (n tokens of it add like n^0.5)
#   2^-22   the exponential, twice: above and below the fraction line
#   cuts    the matrix instructions cut less than a step, 2^-23, off their running sum; two for each
#           tile of 16 tokens, and the sum grows evenly over the 64 of 16 chunks, after which it is
#           put by: 64 / 2 steps at most
#   2^-24   each of the fp32 additions in a row: four a chunk and lane, the joins of lanes, warps, CTAs
# and by the logits' error in log2 units `arg` (of p, above and below).
def step_bound(T, arg=0.0, ctas=152):
    chunks = -(-T // 32 // 12) + 1               # of a warp, if one CTA has them all
    cuts = min(4 * chunks, 64) / 2 + 2
    adds = 4 * chunks + 3 + 12 + min(ctas, chunks)
    return 4 * 2.0 ** -22 + cuts * 2.0 ** -23 + adds * 2.0 ** -24 + 2 * arg


def put_all(pages, table, b, c, codes, s, z, is_v):
    """Codes [T][128], scales and zero points [T][2] of a sequence's KV head into pages."""
    sb, zb = kv4.bf16_bits(s), kv4.bf16_bits(z)
    for t in range(codes.shape[0]):
        kv4.put(pages, table, b, c, t, codes[t], sb[t], zb[t], is_v)


def cache_of(sk, K, V, hq, n_q=1):
    """A cache of one sequence and KV head holding K = (codes, s, z) and V likewise."""
    T = K[0].shape[0]
    mp = -(-T // 64)
    pages = np.zeros((mp, 1, kv4.PAGE_BYTES), np.uint8)
    table = np.arange(mp, dtype=np.int32)[None]
    put_all(pages, table, 0, 0, *K, False)
    put_all(pages, table, 0, 0, *V, True)
    cfg = sk.Config(1, hq, 1, 0, 0, 64)
    cache = sk.Kv4Cache(cfg, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda())
    return cfg, cache, sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q), pages, table


def check_bound(out, lse, ref, tol, lse_tol):
    o, l, bound, _ = ref
    err = np.abs(out.double().cpu().numpy() - o)
    assert np.isfinite(err).all()
    worst = (err / np.maximum(bound, 1e-300)).max()
    assert worst <= tol, f"out: {worst:.3g} of the bound, allowed {tol:.3g}"
    e = np.abs(lse.double().cpu().numpy() - l).max()
    assert e <= lse_tol, f"lse: {e:.3g}, allowed {lse_tol:.3g}"


@pytest.mark.parametrize("hq", [1, 4, 8])
@pytest.mark.parametrize("T", [1, 2, 5, 33, 700, 6000])
def test_attention_of_equal_weights(sk, hq, T):
    """A query of zeros: every weight is the same, exactly, and what is left is the products' error."""
    r = np.random.default_rng(T)
    kv = [(r.integers(0, 16, (T, 128)).astype(np.uint8), r.uniform(0.1, 0.4, (T, 2)).astype(np.float32),
           r.normal(-1, 1, (T, 2)).astype(np.float32)) for _ in range(2)]
    cfg, cache, kws, pages, table = cache_of(sk, *kv, hq)
    q = torch.zeros(1, 1, hq, 128, dtype=torch.bfloat16)
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), 0.1, kws)
    check_bound(out, lse, kv4.attention(q.double().numpy(), pages, table, [T], 0.1), step_bound(T), 2.0 ** -22 * (1 + math.log(T)))


@pytest.mark.parametrize("hq", [4, 8])
def test_attention_of_equal_weights_over_many_chunks(sk, hq):
    """Some 170 chunks a warp of one page, whose even tokens hold the largest codes and odd ones the
    smallest, so that the running sums only grow: without putting them by every 16 chunks the cuts
    alone would come to about 2e-5."""
    B, H, T = 30, 8, 65536
    codes = np.where(np.arange(64)[:, None] % 2 == 0, 15, 0).repeat(128, 1).astype(np.uint8)
    s, z = np.full((64, 2), 0.3125, np.float32), np.full((64, 2), -2.0, np.float32)
    page = np.zeros((1, H, kv4.PAGE_BYTES), np.uint8)
    for c in range(H):
        put_all(page, [[0]], 0, c, codes, s, z, False)
        put_all(page, [[0]], 0, c, codes, s, z, True)
    cfg = sk.Config(B, H * hq, H, 0, 0, 64)
    cache = sk.Kv4Cache(cfg, torch.from_numpy(page).cuda(), torch.zeros(B, T // 64, dtype=torch.int32, device="cuda"))
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    q = torch.zeros(B, 1, H * hq, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = sk.kv4_attention(cfg, cache, q, torch.full((B,), T, dtype=torch.int32, device="cuda"), 0.1, kws)
    bound = 2.0 + 15 * 0.3125
    worst = (out.double() - (-2.0 + 7.5 * 0.3125)).abs().max().item() / bound
    # per warp: 64 / 2 cuts, and 11 times putting by; four additions of zero points a chunk and lane
    tol = 4 * 2.0 ** -22 + 34 * 2.0 ** -23 + (11 + 15 + 152) * 2.0 ** -24 + 4 * 171 / 2 * 2.0 ** -24 * 2.0 / bound
    assert worst <= tol, f"{worst:.3g}, allowed {tol:.3g}"
    assert (lse.double() - math.log(T)).abs().max().item() <= 2.0 ** -20 * math.log(T)


@pytest.mark.parametrize("hq", [3, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_of_whole_number_logits(sk, hq, dtype):
    """Queries and keys whose products are whole numbers: the logits are exact, up to 2^-24 of them in
    the scale, and as much in the exponent."""
    T = 900
    r = np.random.default_rng(3)
    K = (r.integers(0, 16, (T, 128)).astype(np.uint8), np.ones((T, 2), np.float32), np.full((T, 2), -7.0, np.float32))
    V = (r.integers(0, 16, (T, 128)).astype(np.uint8), r.uniform(0.1, 0.4, (T, 2)).astype(np.float32), r.normal(-1, 1, (T, 2)).astype(np.float32))
    cfg, cache, kws, pages, table = cache_of(sk, K, V, hq, 2)
    q = torch.from_numpy(r.integers(-4, 5, (1, 2, hq, 128))).to(DT[dtype])
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), 2.0 ** -6, kws)
    top = 4 * 8 * 128 / 64 * 1.4427            # the largest logit there can be, log2
    arg = 3 * 2.0 ** -24 * top
    check_bound(out, lse, kv4.attention(q.double().numpy(), pages, table, [T], 2.0 ** -6), step_bound(T, arg), arg + 2.0 ** -20)


def scales_case(T, seed, v_scale, k_code=None, k_scale=4.0):
    """K whose first group holds k_code [T][2] in its first two dimensions (times k_scale) and zeros
    elsewhere, the second group random; V of the given scales [T][2], with zero points of its own size."""
    r = np.random.default_rng(seed)
    kc = r.integers(0, 16, (T, 128)).astype(np.uint8)
    kc[:, :64] = 0
    if k_code is not None:
        kc[:, :2] = k_code
    ks, kz = np.tile(np.float32([k_scale, 0.125]), (T, 1)), np.tile(np.float32([0, -1]), (T, 1))
    vz = kv4.bf16_value(kv4.bf16_bits((-8 * v_scale * r.uniform(0.9, 1.1, v_scale.shape)).astype(np.float32)))
    return (kc, ks, kz), (r.integers(0, 16, (T, 128)).astype(np.uint8), v_scale.astype(np.float32), vz)


@pytest.mark.parametrize("hq", [2, 8])
@pytest.mark.parametrize("at", [0, 40, 399])
@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 40, 2.0 ** 100])
def test_attention_beside_a_token_of_large_scale(sk, hq, at, big):
    """A token of very large V, which half of the heads attend to and the others give no weight at
    all (their logit for it is 1200 below): it takes nothing from the others' precision."""
    T = 400
    r = np.random.default_rng(at)
    s = r.uniform(0.1, 0.4, (T, 2))
    s[at] *= big
    code = np.zeros((T, 2), np.uint8)
    code[at, 0] = 15
    K, V = scales_case(T, at + 1, s, code)
    cfg, cache, kws, pages, table = cache_of(sk, K, V, hq)
    q = torch.from_numpy(r.normal(0, 1, (1, 1, hq, 128)) * 0.5).bfloat16()
    q[..., :64] = 0
    q[:, :, :, 0] = torch.where(torch.arange(hq) % 2 == 0, -20.0, 20.0)
    ref = kv4.attention(q.double().numpy(), pages, table, [T], 1.0)
    assert ref[2][0, 0, 0].max() < 100 and ref[2][0, 0, 1].min() > 0.1 * big
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), 1.0, kws)
    # the second group's logits: 64 products of up to 2 and 1, in steps of 2^-19 of 20 (the column's
    # largest) times s for each of four matrix instructions; rounded in fp32 at up to 1200
    arg = 1.4427 * (4 * 2.0 ** -19 * 20 * 0.125 + 3 * 2.0 ** -24 * 1300)
    check_bound(out, lse, ref, step_bound(T, arg), arg + 2.0 ** -20 + 1300 * 2.0 ** -23)


@pytest.mark.parametrize("hq", [1, 8])
def test_attention_groups_and_tokens_of_any_scale(sk, hq):
    """Scales of every size from 2^-60 to 2^60, unrelated in the two groups of dimensions."""
    T = 500
    r = np.random.default_rng(5)
    K, V = scales_case(T, 6, 2.0 ** r.uniform(-60, 60, (T, 2)) * np.float32([1.0, 2.0 ** -50]))
    cfg, cache, kws, pages, table = cache_of(sk, K, V, hq)
    q = torch.zeros(1, 1, hq, 128, dtype=torch.bfloat16)
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), 1.0, kws)
    check_bound(out, lse, kv4.attention(q.double().numpy(), pages, table, [T], 1.0), step_bound(T), 2.0 ** -20 * math.log(T))


@pytest.mark.parametrize("hq", [1, 8])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_attention_weights_against_scales(sk, hq, order):
    """Tokens whose weights fall as their scales rise, from 2^-56 to 2^56: all count alike."""
    T = 480
    r = np.random.default_rng(7)
    e = np.sort(r.integers(0, 15, T))
    e = {"up": e, "down": e[::-1], "mixed": r.permutation(e)}[order]
    code = np.stack([e, np.zeros_like(e)], -1).astype(np.uint8)
    K, V = scales_case(T, 8, r.uniform(1, 2, (T, 2)) * 2.0 ** (8.0 * e[:, None] - 56), code, 8.0)
    cfg, cache, kws, pages, table = cache_of(sk, K, V, hq)
    q = torch.zeros(1, 1, hq, 128, dtype=torch.bfloat16)
    q[..., 0] = -1.0
    scale = math.log(2.0)                       # log2 of the weight: -8 e
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), scale, kws)
    arg = 3 * 2.0 ** -24 * 120
    check_bound(out, lse, kv4.attention(q.double().numpy(), pages, table, [T], float(np.float32(scale))), step_bound(T, arg), arg + 2.0 ** -20 + 2.0 ** -22 * 10)


def test_attention_after_a_token_of_scale_zero_outweighs_all(sk):
    """The reference of the weights moves far up with a token whose scale is 0 (a vector of one value):
    what was summed before it still counts by its own size, here that of all that is in the group."""
    T = 300
    r = np.random.default_rng(9)
    s = r.uniform(0.1, 0.4, (T, 2)) * 2.0 ** 60
    code = np.zeros((T, 2), np.uint8)
    s[150], code[150, 0] = 0.0, 6
    K, V = scales_case(T, 10, s, code, 8.0)
    V[2][150] = 2.0 ** 10
    cfg, cache, kws, pages, table = cache_of(sk, K, V, 2)
    q = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), 1.0, kws)
    arg = 3 * 2.0 ** -24 * 70
    check_bound(out, lse, kv4.attention(q.double().numpy(), pages, table, [T], 1.0), step_bound(T, arg), arg + 2.0 ** -18)


@pytest.mark.parametrize("hq", [2, 8])
@pytest.mark.parametrize("top,scale", [(119, 2.0 ** -6), (127, 2.0 ** -9), (-113, 2.0 ** -6), (-126, 2.0 ** -6)])
def test_attention_of_queries_of_any_size(sk, hq, top, scale):
    """Finite queries far outside f16's range, with keys that make their logits ordinary: whole
    numbers up to 8, times powers of two."""
    T = 300
    r = np.random.default_rng(11)
    unit = 2.0 ** (-top - 2)                     # |q| up to 2^top, |K| up to 8 units, logits up to 2^7 of the scale
    ks = np.tile(np.float32([unit, 1.0]), (T, 1)) if top > 0 else np.full((T, 2), unit, np.float32)
    K = (r.integers(0, 16, (T, 128)).astype(np.uint8), ks, -7 * ks)
    V = (r.integers(0, 16, (T, 128)).astype(np.uint8), r.uniform(0.1, 0.4, (T, 2)).astype(np.float32), r.normal(-1, 1, (T, 2)).astype(np.float32))
    cfg, cache, kws, pages, table = cache_of(sk, K, V, hq)
    q = np.ldexp(r.integers(-8, 9, (1, 1, hq, 128)).astype(np.float64), top - 3)
    q[..., 0], q[..., 64:] = np.ldexp(1.0, top), 0.0
    q = torch.from_numpy(q).bfloat16()
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor([T], dtype=torch.int32).cuda(), scale, kws)
    assert kws.status() == (0, 0)
    arg = 3 * 2.0 ** -24 * 1.4427 * 64 * 2 * scale   # of the largest logit there can be
    check_bound(out, lse, kv4.attention(q.double().numpy(), pages, table, [T], scale), step_bound(T, arg), arg + 2.0 ** -20)


@pytest.mark.parametrize("hq", [1, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("outlier", [0.0, 50.0, 3000.0])
def test_logits_one_by_one(sk, hq, dtype, outlier):
    """Sequences of one token: the log-sum-exp is the logit, held to the header's bound."""
    B, scale = 200, 0.0884
    r = np.random.default_rng(13)
    cfg = sk.Config(B, hq, 1, 0, 0, 64)
    pages, table = np.zeros((B, 1, kv4.PAGE_BYTES), np.uint8), np.arange(B, dtype=np.int32)[:, None]
    for b in range(B):
        s, z = r.uniform(0.05, 2, (1, 2)), r.normal(-3, 3, (1, 2))
        put_all(pages, table, b, 0, r.integers(0, 16, (1, 128)).astype(np.uint8), s.astype(np.float32), z.astype(np.float32), False)
    cache = sk.Kv4Cache(cfg, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda())
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    q = r.normal(0, 1, (B, 1, hq, 128))
    for i in range(B):
        q[i, 0, :, r.integers(0, 128)] += outlier
    q = torch.from_numpy(q).to(DT[dtype])
    _, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.ones(B, dtype=torch.int32, device="cuda"), scale, kws)
    scale = float(np.float32(scale))
    want = kv4.attention(q.double().numpy(), pages, table, [1] * B, scale)
    q = np.abs(q.double().numpy())[:, 0]
    s = np.stack([kv4.bf16_value(pages[:, 0, 2048 + 4 * g:2050 + 4 * g].copy().view(np.uint16)[:, 0]) for g in range(2)], 1).astype(np.float64)
    z = np.stack([kv4.bf16_value(pages[:, 0, 2050 + 4 * g:2052 + 4 * g].copy().view(np.uint16)[:, 0]) for g in range(2)], 1).astype(np.float64)
    size = np.einsum("bhgd,bg->bh", q.reshape(B, hq, 2, 64), np.abs(z) + 15 * s)
    bound = scale * (2.0 ** -16 * q.max(-1) * s.sum(1)[:, None] + 2.0 ** -22 * size)
    # the way to log2 and back: 2^-22 of the logit
    err = np.abs(lse.double().cpu().numpy() - want[1])[:, 0]
    assert (err <= bound + 2.0 ** -22 * np.abs(want[1][:, 0])).all(), (err / bound).max()


# ------------------------------------------------------------------ the 4-bit cache's codes
def rows_at_halves(dtype):
    """Groups of 64 for every significand of a scale s and every half n + 1/2: the dividend x - z is
    that half times s, exactly, and next to it by one step of fp32 and by more; and the ends of
    the range.  (z takes all of the half's bits that bf16 holds, x the rest and the step.)"""
    groups = []
    to = lambda v: torch.tensor(v, dtype=torch.float32).to(DT[dtype]).float().tolist()  # noqa: E731
    for m in range(128, 256):
        s = m / 64.0
        for n in range(15):
            half = (n + 0.5) * s
            z = kv4.bf16_value(kv4.bf16_floor_bits(np.float32(-half))).item()
            step = 2.0 ** (math.floor(math.log2(half)) - 23)
            rest = half + z
            xs = [rest + k * step / 2 for k in range(-8, 9)] + [rest * (1 + k / 256) for k in range(-10, 11)]
            xs += [z + (n + h) * s for h in (0.4, 0.499, 0.5, 0.501, 0.6)] + [z + i * s for i in range(16)]
            xs = [min(max(x, z), z + 15 * s) for x in to(xs)]
            groups.append((to([z, z + 15 * s]) + xs + [z] * 64)[:64])
    return torch.tensor(groups).view(-1, 128)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_codes_of_dividends_at_every_half(sk, dtype):
    """The codes come from a corrected reciprocal; they are those of a division."""
    x = rows_at_halves(dtype).to(DT[dtype])[None, :, None]
    T = x.shape[1]
    mp = -(-T // 64)
    cfg = sk.Config(1, 1, 1, 0, 0, 64)
    table = np.arange(mp, dtype=np.int32)[None]
    cache = sk.Kv4Cache(cfg, torch.zeros(mp, 1, 9216, dtype=torch.uint8, device="cuda"), torch.from_numpy(table).cuda())
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    sk.kv4_append(cfg, cache, x.cuda(), (-x).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), kws)
    want = np.zeros((mp, 1, kv4.PAGE_BYTES), np.uint8)
    for is_v, y in ((0, x), (1, -x)):
        n, sb, zb = kv4.quantise(y.float().numpy())
        if not is_v:
            assert len(set((sb & 127).reshape(-1).tolist())) == 128   # every significand of a scale
        for t in range(T):
            kv4.put(want, table, 0, 0, t, n[0, t, 0], sb[0, t, 0], zb[0, t, 0], is_v)
    assert np.array_equal(cache.pages.cpu().numpy(), want)


# ------------------------------------------------------------------ together
def step_inputs(sk, B=2, hq=8, hkv=2, V=3000):
    cfg = sk.Config(B, hq, hkv, 0, 0, 64)
    mp = 4
    pages = torch.zeros(B * mp, hkv, 9216, dtype=torch.uint8, device="cuda")
    cache = sk.Kv4Cache(cfg, pages, torch.arange(B * mp, dtype=torch.int32, device="cuda").view(B, mp))
    g = gen(21)
    x = {n: torch.randn(B, 1, h, 128, generator=g).bfloat16().cuda() for n, h in (("q", hq), ("k", hkv), ("v", hkv))}
    x["logits"], x["tok"] = torch.randn(B, V, generator=g).cuda(), torch.tensor([3, V - 1]).cuda()
    return cfg, cache, x, sk.RopePlan(128)


def test_a_step_captured_over_two_streams(sk, ws):
    """Calls that fork and join inside one captured graph: launches that may start early only do so
    behind the kernel before them on their own stream, and all wait for what they need."""
    cfg, cache, x, plan = step_inputs(sk)
    B = cfg.batch
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    first, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    one, H = torch.zeros(B, 1, dtype=torch.int64, device="cuda"), torch.full((B, 1), 9.0, device="cuda")
    side = torch.cuda.Stream()

    def step(fork):
        s = side if fork else None
        here = torch.cuda.current_stream()
        qr, kr = sk.rope(plan, x["q"], x["k"], pos)
        if fork:
            side.wait_stream(here)
        sk.kv4_append(cfg, cache, kr, x["v"], first, kws, stream=s)
        r = sk.token_logprobs(x["logits"], x["tok"], ws, n_top=3)
        H.fill_(9)
        sk.surprisal(x["logits"][:, None], one, ws, out=H)      # a fill, no kernel of its own
        if fork:
            here.wait_stream(side)
        o, lse = sk.kv4_attention(cfg, cache, qr, lens, 0.0884, kws)
        return [o, lse, r.logprob, r.top_ids, H.clone()]

    def set_step(t):
        pos.fill_(t); first.fill_(t); lens.fill_(t + 1)
        for i, n in enumerate(("q", "k", "v", "logits")):
            x[n].copy_(torch.randn(x[n].shape, generator=gen(100 * t + i)))
    set_step(0)
    step(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(True)
    want = []
    cache.pages.zero_()
    for t in range(60):
        set_step(t)
        want.append([a.clone() for a in step(False)])
        torch.cuda.synchronize()
    cache.pages.zero_()
    for t in range(60):
        set_step(t)
        graph.replay()
        for a, b in zip(got, want[t]):
            assert torch.equal(a, b), t
    assert kws.status() == (0, 0) and ws.status() == (0, 0)


def test_calls_from_two_threads(sk):
    """Two host threads, each with its own stream, workspaces and cache."""
    import threading
    results = [None, None]

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            cfg, cache, x, plan = step_inputs(sk)
            w, kws = sk.Workspace(cfg), sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
            out = []
            for t in range(100):
                i32 = dict(dtype=torch.int32, device="cuda")
                qr, kr = sk.rope(plan, x["q"], x["k"], torch.full((1,), t, **i32))
                sk.kv4_append(cfg, cache, kr, x["v"], torch.full((2,), t, **i32), kws)
                o, _ = sk.kv4_attention(cfg, cache, qr, torch.full((2,), t + 1, **i32), 0.1, kws)
                out += [o, sk.token_logprobs(x["logits"], x["tok"], w, n_top=2).top_logprobs]
            results[i] = [a.cpu() for a in out] + [kws.status(), w.status()]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert results[0][-2:] == results[1][-2:] == [(0, 0), (0, 0)]
    for a, b in zip(results[0][:-2], results[1][:-2]):
        assert torch.equal(a, b)


def test_rows_further_apart_than_32_bits(sk, ws):
    """Sequences 2^32 and more elements apart, in and out."""
    far = (1 << 32) + 1024
    big = torch.empty(far + 65536, dtype=torch.bfloat16, device="cuda")
    T, H = 20, 3
    x = big.as_strided((2, T, H, 128), (far, H * 128, 128, 1))
    x.copy_(torch.randn(2, T, H, 128, generator=gen(1)))
    near = x.clone()
    plan, pos = sk.RopePlan(128), torch.arange(T, dtype=torch.int32, device="cuda")
    want = sk.rope(plan, near, None, pos)[0]
    assert torch.equal(sk.rope(plan, x, None, pos)[0], want)
    cfg = sk.Config(2, H, H, 0, 0, 64)
    caches = [sk.Kv4Cache(cfg, torch.zeros(2, H, 9216, dtype=torch.uint8, device="cuda"),
                          torch.arange(2, dtype=torch.int32, device="cuda").view(2, 1)) for _ in range(2)]
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    for c, y in zip(caches, (near, x)):
        sk.kv4_append(cfg, c, y, y, zero, kws)
    assert torch.equal(caches[0].pages, caches[1].pages)
    logits = big.as_strided((2, 4, 1999), (far, 2048, 1))
    logits.copy_(torch.randn(2, 4, 1999, generator=gen(2)))
    tok = torch.randint(0, 1999, (2, 4), generator=gen(3)).cuda()
    r = sk.token_logprobs(logits, tok, ws, n_top=5)
    want_lp = tokens.token_logprobs(logits.double().cpu().numpy().reshape(8, 1999), tok.cpu().numpy().reshape(-1), 1.0, 5)
    assert np.array_equal(r.top_ids.cpu().numpy().reshape(8, 5), want_lp["top_ids"])
    # not bit for bit a call on rows of 1999 side by side: those start at other offsets in their
    # 16-byte vectors, and so group their sums otherwise.  Exponents of up to 10, 2000 / 128 + 40 additions,
    # the result's own size (up to 13)
    d = 30 * 2.0 ** -24 + 2.0 ** -22 + 56 * 2.0 ** -24
    for name in ("logprob", "lse", "entropy", "top_logprobs"):
        got = getattr(r, name).double().cpu().numpy().reshape(want_lp[name].shape)
        assert np.abs(got - want_lp[name]).max() <= 3 * d * (14 if name == "entropy" else 1) + 2.0 ** -22 * 13, name
    x.copy_(near)
    sk.rope(plan, x, None, pos, q_out=x)
    assert torch.equal(x, want)
    assert kws.status() == (0, 0) and ws.status() == (0, 0)


def test_most_sequences_a_cache_may_have(sk):
    """1024 sequences, half of them empty, over pages that they share."""
    B, H, hq, T = 1024, 2, 6, 150
    cfg1, one, ws1 = small_cache(sk, 1, H, hq, T, seed=4)
    cfg = sk.Config(B, hq, H, 0, 0, 64)
    cache = sk.Kv4Cache(cfg, one.pages, one.page_table.repeat(B, 1))
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=2)
    lens = torch.randint(0, T + 1, (B,), generator=gen(2)).int()
    lens[::2] = 0
    q = torch.randn(B, 2, hq, 128, generator=gen(3)).bfloat16()
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), lens.cuda(), 0.0884, kws)
    assert kws.status() == (0, 0)
    assert not out[::2].any() and (lse[::2] == -INF).all()
    pages, table = one.pages.cpu().numpy(), one.page_table.cpu().numpy()
    scale = float(np.float32(0.0884))
    for b in (1, 37, 511, 1023):
        ref = kv4.attention(q[b:b + 1].double().numpy(), pages, table, [int(lens[b])], scale)
        # scales below 0.5, |q| below 5, |K| below 5: what the header allows a logit
        arg = 1.4427 * scale * (2.0 ** -16 * 5 * 1 + 2.0 ** -22 * 128 * 5 * 10)
        check_bound(out[b:b + 1], lse[b:b + 1], ref, step_bound(T, arg), arg + 2.0 ** -20)


def test_append_of_one_row_for_all_tokens_and_more_valid_than_there_are(sk):
    """Rows of k and v may lie on one another; n_valid beyond the rows counts as all of them."""
    cfg, cache, kws = small_cache(sk, 2, 2, 2, 128)
    _, other, _ = small_cache(sk, 2, 2, 2, 128)
    k, v = (torch.randn(2, 1, 2, 128, generator=gen(i)).half().cuda() for i in range(2))
    first = torch.tensor([3, 60], dtype=torch.int32).cuda()
    sk.kv4_append(cfg, cache, k.expand(2, 40, 2, 128), v.expand(2, 40, 2, 128), first, kws, n_valid=first * 0 + 1000)
    sk.kv4_append(cfg, other, k.repeat(1, 40, 1, 1), v.repeat(1, 40, 1, 1), first, kws)
    assert torch.equal(cache.pages, other.pages)
    a, b = sk.kv4_read(cfg, cache, first, 40, kws, n_valid=first * 0 + 41), sk.kv4_read(cfg, cache, first, 40, kws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and kws.status() == (0, 0)


def test_a_million_short_rows(sk, ws):
    x = torch.randn(1 << 20, 50, generator=gen(1)).bfloat16()
    tok = torch.randint(0, 50, (1 << 20,), generator=gen(2))
    r = sk.token_logprobs(x.cuda(), tok.cuda(), ws, n_top=2)
    want = torch.log_softmax(x.double(), -1)
    # exponents of up to 13 with three roundings, 2^-22 of the exponential, 8 + 7 additions: 58 * 2^-24
    assert (r.logprob.cpu().double() - want.gather(1, tok[:, None])[:, 0]).abs().max().item() <= 2.0 ** -18
    ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(r.top_ids.cpu().long(), ids)
