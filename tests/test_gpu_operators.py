"""GPU parity of the token operators (log-probabilities, surprisal, rotary
positions) and of the 4-bit cache against their fp64 oracles."""
import math

import numpy as np
import pytest
import torch

from oracle import kv4, tokens

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "f32": 2.0 ** -24}   # half a step, relative
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
def check_logprobs(r, ref, scale, span, vocab):
    """span: largest |scale (x - max)| that still counts (e^-100 of a sum does not).  Rounding:
    the argument of each exponential errs by 3 * 2^-24 * min(span, 100), the exponential
    by 2^-22, the sum's additions (one chain per thread, then a tree) by 2^-24 each; the
    values themselves by 2^-23 of their size, and by 2^-23 of the logit products."""
    d = 3 * 2.0 ** -24 * min(span, 100) + 2.0 ** -22 + 2.0 ** -24 * (vocab / 512 + 40)
    for name in ("logprob", "lse", "entropy"):
        got, want = getattr(r, name).double().cpu().numpy().reshape(-1), ref[name]
        extra = (1 + abs(want)) if name == "entropy" else 1.0  # the mean of x - max moves by d times its size too
        compare(got, want, 3 * d * extra + 2.0 ** -22 * (np.abs(np.where(np.isfinite(want), want, 0)) + span * (name != "entropy")), name)
    if r.top_ids is not None:
        assert np.array_equal(r.top_ids.cpu().numpy().reshape(ref["top_ids"].shape), ref["top_ids"])
        compare(r.top_logprobs.double().cpu().numpy().reshape(ref["top_ids"].shape), ref["top_logprobs"], 3 * d + 2.0 ** -21 * span, "top")


def compare(got, want, tol, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    fin = np.isfinite(want)
    other = ~fin & ~np.isnan(want)
    assert np.array_equal(got[other], want[other]), what
    assert np.isfinite(got[fin]).all(), what
    err = np.abs(got[fin] - want[fin])
    tol = np.broadcast_to(tol, want.shape)[fin]
    assert (err <= tol).all(), f"{what}: error {err.max():.3g}, allowed {tol[err.argmax()]:.3g}"


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 7, 32), (2, 33, 5), (5, 511, 32), (2, 4097, 1), (1, 20011, 20),
                                            (40, 4099, 7), (400, 600, 3)])
def test_logprobs(sk, ws, dtype, rows, vocab, top):
    g = gen(rows * 7 + vocab)
    x = (torch.randn(rows, vocab, generator=g) * 4).to(DT[dtype])
    tok = torch.randint(0, vocab, (rows,), generator=g)
    tok[0] = vocab - 1
    r = sk.token_logprobs(x.cuda(), tok.cuda(), ws, n_top=top, scale=0.75)
    ref = tokens.token_logprobs(x.double().numpy(), tok.numpy(), 0.75, top)
    check_logprobs(r, ref, 0.75, float(0.75 * (x.max() - x.min()).float() + 0.75 * x.abs().max().float()), vocab)
    assert ws.status() == (0, 0)
    # the same without the extras, and with 32-bit ids
    r2 = sk.token_logprobs(x.cuda(), tok.int().cuda(), ws, scale=0.75, entropy=False)
    assert r2.lse is None and r2.top_ids is None and torch.equal(r2.logprob, r.logprob)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_strides_and_alignment(sk, ws, dtype):
    """[B][T][V] cut out of a wider, longer buffer whose rows start at odd elements."""
    g = gen(5)
    big = (torch.randn(2, 4, 1003, generator=g) * 3).to(DT[dtype]).cuda()
    x = big[:, 1:4, 3:804]
    tok = torch.randint(0, 801, (2, 5), generator=g).cuda()[:, 1:4]
    r = sk.token_logprobs(x, tok, ws, n_top=4)
    ref = tokens.token_logprobs(x.double().cpu().numpy().reshape(6, 801), tok.cpu().numpy().reshape(-1), 1.0, 4)
    assert r.logprob.shape == (2, 3) and r.top_ids.shape == (2, 3, 4)
    check_logprobs(r, ref, 1.0, float(2 * (x.max() - x.min())), 801)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
def test_logprobs_masked_and_special_rows(sk, ws, dtype):
    low = torch.finfo(DT[dtype]).min
    V = 1500
    x = torch.randn(9, V, generator=gen(6)).to(DT[dtype])
    x[0, 3:] = -INF                 # three entries left, the token among them
    x[1] = -INF                     # nothing left
    x[2] = low                      # all at the type's lowest value: uniform
    x[3, 10:] = low
    x[4, 700] = math.nan
    x[5, 1499] = INF
    x[6] = 0.0                      # all alike
    x[6, ::2] = -0.0
    x[7, :] = -INF
    x[7, 1400] = low                # one entry left, of the lowest value
    tok = torch.tensor([2, 0, 7, 5, 1, 1, 1499, 1400, -1])
    r = sk.token_logprobs(x.cuda(), tok.cuda(), ws, n_top=5)
    ref = tokens.token_logprobs(x.double().numpy(), tok.numpy(), 1.0, 5)
    # lse near the lowest value is held to fp32's step there
    for i in range(9):
        one = sk.TokenLogprobs(*[t[i:i + 1] for t in r])
        span = 0.0 if i in (2, 7) else 20.0
        sub = {k: v[i:i + 1] for k, v in ref.items()}
        check_logprobs(one, sub, 1.0, span, V)
    assert ws.status() == (0, 0)


@pytest.mark.parametrize("scale,offset", [(1e-3, 0.0), (0.02, 0.0), (30.0, 0.0), (2000.0, 0.0), (1.0, 3000.0), (1.0, 60000.0), (1.0, -1e6)])
def test_logprobs_scales_and_offsets(sk, ws, scale, offset):
    """Very flat and very sharp distributions; logits with a large common offset, whose
    log-probabilities are those without it (the logits of f32 being rounded first)."""
    x = torch.randn(5, 9001, generator=gen(1)) * 3 + offset
    tok = x.argmax(1)
    r = sk.token_logprobs(x.cuda(), tok.cuda(), ws, n_top=6, scale=scale)
    ref = tokens.token_logprobs(x.double().numpy(), tok.numpy(), float(np.float32(scale)), 6)
    assert np.array_equal(r.top_ids.cpu().numpy(), ref["top_ids"])
    # exponents err by 3 * 2^-24 of what still counts (100) and 2^-22, sums by 2^-24 an addition
    d = 300 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -24 * (9001 / 256 + 40)
    for name in ("logprob", "top_logprobs", "entropy"):
        want = ref[name]
        compare(getattr(r, name).double().cpu().numpy(), want, 3 * d * (1 + np.abs(want)), name)
    compare(r.lse.double().cpu().numpy(), ref["lse"], 3 * d + 2.0 ** -22 * np.abs(ref["lse"]), "lse")


def test_logprobs_bad_token_is_flagged(sk, ws):
    x = torch.zeros(3, 50, device="cuda")
    r = sk.token_logprobs(x, torch.tensor([1, 50, -1]).cuda(), ws)
    lp = r.logprob.tolist()
    assert abs(lp[0] + math.log(50)) < 1e-5 and math.isnan(lp[1]) and lp[2] == 0
    assert ws.status() == (1, 1)
    r = sk.token_logprobs(x, torch.tensor([1, -2, -1]).cuda(), ws)
    assert math.isnan(r.logprob[1].item()) and ws.status() == (1, 1)


@pytest.mark.parametrize("vocab", [3000, 60000])
def test_logprobs_ties_and_crowded_alternatives(sk, ws, vocab):
    """Alternatives among many equal logits, in sorted rows, and all in the vectors of a
    single thread (more candidates than the kernel keeps)."""
    x = torch.zeros(6, vocab)
    x[1] = torch.arange(vocab) // 100 % 7       # ties everywhere
    x[2] = -torch.arange(vocab, dtype=torch.float32)
    x[3] = torch.arange(vocab, dtype=torch.float32)
    x[4] = (torch.arange(vocab) % 4096 < 8).float() * (1 + torch.arange(vocab) / vocab)
    x[5] = ((torch.arange(vocab) // 4) % 512 == 5).float() * (2 + torch.arange(vocab) / vocab)
    tok = torch.zeros(6, dtype=torch.int64)
    r = sk.token_logprobs(x.cuda(), tok.cuda(), ws, n_top=32)
    ref = tokens.token_logprobs(x.double().numpy(), tok.numpy(), 1.0, 32)
    assert np.array_equal(r.top_ids.cpu().numpy(), ref["top_ids"])


def test_logprobs_more_candidates_than_places(sk, ws):
    """Enough rows that one CTA has a whole row, whose largest logits all lie in the vectors
    of eight threads: about 900 candidates for 32 places."""
    V = 60000
    i = torch.arange(V)
    x = ((i // 4) % 512 < 8).float() * (2 + (i * 7919 % V) / V)
    ref = tokens.token_logprobs(x[None].double().numpy(), [5], 1.0, 32)
    tok = torch.full((320,), 5, dtype=torch.int64, device="cuda")
    r = sk.token_logprobs(x.cuda().expand(320, V), tok, ws, n_top=32)
    assert (r.top_ids.cpu().numpy() == ref["top_ids"]).all()
    check_logprobs(sk.TokenLogprobs(*[t[300:301] for t in r]), ref, 1.0, 4.0, V)


@pytest.mark.parametrize("B,T,V", [(1, 1, 50), (1, 2, 300), (3, 9, 1001), (2, 40, 20000)])
def test_surprisal(sk, ws, B, T, V):
    g = gen(T)
    x = (torch.randn(B, T, V, generator=g) * 3).bfloat16()
    tok = torch.randint(0, V, (B, T), generator=g)
    tok[-1, -1] = -1
    H = sk.surprisal(x.cuda(), tok.cuda(), ws)
    ref = tokens.surprisal(x.double().numpy(), tok.numpy())
    compare(H.double().cpu().numpy(), ref, 2.0 ** -22 * 60 + 2.0 ** -24 * (V / 512 + 60), "H")
    # into a given buffer, token ids in 32 bits, logits of the last position never read
    x[:, -1] = math.nan
    H2 = torch.full((B, T), 7.0, device="cuda")
    sk.surprisal(x.cuda(), tok.int().cuda(), ws, out=H2)
    assert torch.equal(H, H2)


# ------------------------------------------------------------------ rotary positions
def rope_case(sk, dtype, B, T, hq, hkv, D, rot, inter, scaling, seed, far=2000):
    g = gen(seed)
    q = torch.randn(B, T, hq, D, generator=g).to(DT[dtype])
    k = torch.randn(B, T, hkv, D, generator=g).to(DT[dtype])
    pos = torch.randint(0, far, (B, T), generator=g)
    plan = sk.RopePlan(rot, 500000.0, inter, scaling, 8.0, 4096)
    f, m = tokens.rope_frequencies(rot, 500000.0, scaling, 8.0, 4096)
    return q, k, pos, plan, f, m


def check_rope(got, x, pos, f, m, inter, dtype, backward=False):
    """Half a step of the type, and the fp32 products: the angle errs by 2^-24 of a half
    turn, sine and cosine by 2^-23, two products and a sum by 2^-24 each."""
    want = tokens.rope(x.double().numpy(), pos.numpy(), f, m, inter, backward)
    size = np.abs(x.double().numpy()).max() * m
    compare(got.double().cpu().numpy(), want, HALF[dtype] * np.abs(want) + 2.0 ** -20 * size, "rope")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,T,hq,hkv,D,rot,scaling", [
    (1, 1, 32, 8, 128, 128, "banded"), (2, 5, 7, 1, 128, 64, "parts"), (3, 2, 2, 1, 96, 24, "linear"),
    (1, 3, 1, 1, 10, 6, "none"), (2, 700, 4, 2, 64, 64, "ntk"), (1, 1, 3, 5, 257, 2, "none"), (1, 2, 1, 1, 1024, 512, "none")])
def test_rope(sk, dtype, inter, B, T, hq, hkv, D, rot, scaling):
    q, k, pos, plan, f, m = rope_case(sk, dtype, B, T, hq, hkv, D, rot, inter, scaling, D + T)
    qo, ko = sk.rope(plan, q.cuda(), k.cuda(), pos.cuda())
    check_rope(qo, q, pos, f, m, inter, dtype)
    check_rope(ko, k, pos, f, m, inter, dtype)
    assert torch.equal(qo[..., rot:].cpu(), q[..., rot:])
    # queries alone, 32-bit positions, in place
    q2 = q.cuda()
    sk.rope(plan, q2, None, pos.int().cuda(), q_out=q2)
    assert torch.equal(q2, qo)
    # keys alone, turned the other way
    kb = sk.rope(plan, None, k.cuda(), pos.cuda(), backward=True)[1]
    check_rope(kb, k, pos, f, m, inter, dtype, True)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_far_positions(sk, inter):
    """Positions up to 2^40: the angle keeps its fraction of a turn.  The oracle's own fp64
    product is taken modulo one turn in exact integers."""
    q, k, pos, plan, f, m = rope_case(sk, "f32", 1, 6, 2, 1, 64, 64, inter, "none", 3)
    pos[0] = torch.tensor([0, 1 << 20, (1 << 31) - 1, 1 << 33, (1 << 40) - 7, 12345678901])
    from decode_attention_span_gb300 import rotary
    freqs = [int(v) % (1 << 64) for v in rotary.rope_freqs(plan.config)[0]]
    got = sk.rope(plan, q.cuda(), None, pos.cuda())[0].double().cpu().numpy()
    for t in range(6):
        ang = np.array([(int(pos[0, t]) * u % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for u in freqs])
        want = tokens.rope(q[:, t:t + 1].double().numpy(), [[1]], ang, 1.0, inter)
        compare(got[:, t:t + 1], want, 2.0 ** -20 * 5, f"token {t}")


def test_rope_strides_padding_and_layout(sk):
    """Heads cut out of one projection, keys written to [B][Hkv][T][D], a padded batch whose
    padding keeps what the output held, positions shared by the batch."""
    B, T, D = 2, 6, 128
    g = gen(9)
    qkv = torch.randn(B, T, 4 + 2 + 2, D, generator=g).bfloat16().cuda()
    q, k = qkv[:, :, :4], qkv[:, :, 4:6]
    pos = torch.arange(T).repeat(B, 1)
    pos[1, 4:] = -1
    plan = sk.RopePlan(D)
    f, m = tokens.rope_frequencies(D, 10000.0)
    K = torch.full((B, 2, T, D), 5.0, dtype=torch.bfloat16, device="cuda")
    qo, ko = sk.rope(plan, q, k, pos.cuda(), k_out=K.transpose(1, 2))
    assert ko.data_ptr() == K.data_ptr()
    qw, kw = q.cpu().clone(), k.cpu().clone()
    qw[1, 4:], kw[1, 4:] = 0, 5.0
    check_rope(qo, qw, pos, f, m, False, "bf16")
    check_rope(K.transpose(1, 2), kw, pos, f, m, False, "bf16")
    before = qkv.clone()
    sk.rope(plan, q, k, torch.arange(T).cuda(), q_out=q, k_out=k)   # in place in the projection's rows
    assert torch.equal(qkv[:, :, 6:], before[:, :, 6:])
    check_rope(q, before[:, :, :4].cpu(), torch.arange(T).repeat(B, 1), f, m, False, "bf16")


def test_rope_gradient(sk):
    """backward=True is the transpose: <dy, rope(x)> = <rope'(dy), x>, and the gradient agrees
    with differences of the forward call."""
    q, k, pos, plan, f, m = rope_case(sk, "f32", 2, 3, 2, 1, 64, 32, False, "parts", 4)
    dy = torch.randn(q.shape, generator=gen(1)).cuda()
    dx = sk.rope(plan, dy, None, pos.cuda(), backward=True)[0]
    dot = lambda a, b: (a.double() * b.double()).sum().item()  # noqa: E731
    fwd = lambda x: sk.rope(plan, x, None, pos.cuda())[0]      # noqa: E731
    x = q.cuda()
    # sums of 768 products of size up to 16 m, each rounded once or twice in fp32
    assert abs(dot(dy, fwd(x)) - dot(dx, x)) < 768 * 16 * m * 2.0 ** -21
    step = torch.randn(q.shape, generator=gen(2)).cuda()
    diff = (dot(dy, fwd(x + step)) - dot(dy, fwd(x - step))) / 2  # linear: exact but for rounding
    assert abs(diff - dot(dx, step)) < 768 * 40 * m * 2.0 ** -21


# ------------------------------------------------------------------ the 4-bit cache
def kv_cache(sk, B, Hkv, max_pages, n_q=1, hq=None, seed=0):
    cfg = sk.Config(B, hq or Hkv, Hkv, 0, 0, 64)
    n = B * max_pages + 2
    g = gen(seed)
    pages = torch.randint(0, 256, (n, Hkv, 9216), dtype=torch.uint8, generator=g)  # old contents: anything
    table = torch.randperm(n, generator=g)[:B * max_pages].int().view(B, max_pages)
    return cfg, sk.Kv4Cache(cfg, pages.cuda(), table.cuda().contiguous()), sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q)


def kv_rows(dtype, B, T, H, seed):
    g = gen(seed)
    ch = torch.where(torch.rand(H, 128, generator=g) < 0.1, 8.0, 1.0)
    k = (torch.randn(B, T, H, 128, generator=g) * ch + torch.randn(H, 128, generator=g) * ch).to(DT[dtype])
    return k, torch.randn(B, T, H, 128, generator=g).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,H,T,first,valid", [
    (1, 1, 1, [0], None), (2, 3, 1, [63, 64], None), (2, 2, 70, [5, 0], None), (3, 2, 33, [0, 17, 100], [33, 0, 20]),
    (1, 8, 200, [16], None), (1, 4, 128, [64], [128])])
def test_kv4_append_writes_the_documented_bytes(sk, dtype, B, H, T, first, valid):
    cfg, cache, ws = kv_cache(sk, B, H, 5, seed=T)
    k, v = kv_rows(dtype, B, T, H, T + 1)
    k[0, 0, 0, 5:64] = k[0, 0, 0, 5]       # nearly constant, and constant groups
    v[0, T - 1, H - 1, 64:] = 0.25
    want = cache.pages.cpu().numpy().copy()
    table = cache.page_table.cpu().numpy()
    for is_v, x in ((0, k), (1, v)):
        n, sb, zb = kv4.quantise(x.float().numpy())
        for b in range(B):
            for t in range(T if valid is None else valid[b]):
                for c in range(H):
                    kv4.put(want, table, b, c, first[b] + t, n[b, t, c], sb[b, t, c], zb[b, t, c], is_v)
    f = torch.tensor(first, dtype=torch.int32).cuda()
    nv = None if valid is None else torch.tensor(valid, dtype=torch.int32).cuda()
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), f, ws, n_valid=nv)
    assert ws.status() == (0, 0)
    assert np.array_equal(cache.pages.cpu().numpy(), want)   # every other byte as it was
    # read back: z + s n rounded to each type; rows past n_valid as they were
    for out_t in ("bf16", "fp16", "f32"):
        out = [torch.full((B, H, T, 128), 3.0, dtype=DT[out_t], device="cuda") for _ in range(2)]
        sk.kv4_read(cfg, cache, f, T, ws, n_valid=nv, out=out)
        for is_v, x, y in ((0, k, out[0]), (1, v, out[1])):
            n, sb, zb = kv4.quantise(x.float().numpy())
            ref = kv4.values(n, sb, zb).transpose(0, 2, 1, 3).copy()
            if valid is not None:
                for b in range(B):
                    ref[b, :, valid[b]:] = 3.0
            # one rounding to fp32, one to the type; f16 loses to its smallest step near 0
            tol = (HALF[out_t] + 2.0 ** -24) * np.abs(ref) + (2.0 ** -25 if out_t == "fp16" else 0)
            compare(y.double().cpu().numpy(), ref, tol, "read")
    kd, vd = sk.kv4_read(cfg, cache, f, T, ws)
    assert kd.dtype == torch.bfloat16 and kd.shape == (B, H, T, 128) and ws.status() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_kv4_append_ties_and_tiny_steps(sk, dtype):
    """Whole numbers whose quotients fall on halves (to the even code), for every step from 2
    to 16 and for steps of powers of two down to where they vanish, and steps below 2^-100."""
    cfg, cache, ws = kv_cache(sk, 1, 1, 2)
    x = torch.zeros(60, 128)
    for r in range(15):                      # s = r + 2: values 0, s / 2, s, ... 15 s
        x[r, :64] = (torch.arange(64) % 31) * (r + 2) / 2
        x[r, 64:] = -x[r, :64]
    for r in range(15, 60):
        x[r, :64] = (torch.arange(64) % 31) * 2.0 ** -(r * 2.9 // 1 + (0 if dtype == "bf16" else -40))
        x[r, 64:] = x[r, :64] * (1 + 2.0 ** -5)
    x = x.to(DT[dtype])[None, :, None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, x.cuda(), -x.cuda(), zero, ws)
    want = cache.pages.cpu().numpy().copy()
    table = cache.page_table.cpu().numpy()
    for is_v, y in ((0, x), (1, -x)):
        n, sb, zb = kv4.quantise(y.float().numpy())
        for t in range(60):
            kv4.put(want, table, 0, 0, t, n[0, t, 0], sb[0, t, 0], zb[0, t, 0], is_v)
    assert np.array_equal(cache.pages.cpu().numpy(), want)


def test_kv4_append_strides_and_non_finite(sk):
    cfg, cache, ws = kv_cache(sk, 2, 2, 2)
    g = gen(3)
    qkv = torch.randn(2, 20, 4 + 2 + 2, 128, generator=g).bfloat16()
    qkv[0, 3, 4, 10], qkv[1, 4, 7, 100], qkv[1, 5, 6, 0] = math.nan, INF, -INF
    qkv = qkv.cuda()
    first = torch.zeros(2, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, qkv[:, :, 4:6], qkv[:, :, 6:], first, ws)
    kd, vd = sk.kv4_read(cfg, cache, first, 20, ws, dtype=torch.float32)
    for x, y in ((qkv[:, :, 4:6], kd), (qkv[:, :, 6:], vd)):
        n, sb, zb = kv4.quantise(x.float().cpu().numpy())
        ref = kv4.values(n, sb, zb).transpose(0, 2, 1, 3)
        compare(y.double().cpu().numpy(), ref, 2.0 ** -24 * np.abs(ref), "read")
    assert torch.isnan(kd[0, 0, 3, :64]).all() and torch.isfinite(kd[0, 0, 3, 64:]).all()
    assert torch.isnan(vd[1, 1, 4, 64:]).all() and torch.isnan(vd[1, 0, 5, :64]).all()


def test_kv4_bad_pages_and_positions_are_flagged(sk):
    """A page id out of range or a position past the table: that token is not stored, not
    read and not attended to, the others are, and the workspace names the sequence."""
    cfg, cache, ws = kv_cache(sk, 2, 1, 2)
    table = cache.page_table.clone()
    k, v = kv_rows("bf16", 2, 70, 1, 0)
    first = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 1, 1, 128, generator=gen(1)).bfloat16().cuda()
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), first, ws)
    full = sk.kv4_attention(cfg, cache, q, torch.tensor([70, 64], dtype=torch.int32).cuda(), 0.1, ws)
    assert ws.status() == (0, 0)
    for bad in (-1, cache.pages.shape[0], 1 << 30):
        cache.page_table.copy_(table)
        cache.page_table[1, 1] = bad
        sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), first, ws)
        assert ws.status() == (1, 1)
        out = [torch.full((2, 1, 70, 128), 9.0, device="cuda") for _ in range(2)]
        sk.kv4_read(cfg, cache, first, 70, ws, out=out)
        assert ws.status() == (1, 1)
        assert (out[0][1, 0, 64:] == 9.0).all() and (out[0][1, 0, :64] != 9.0).any(-1).all()
        o, lse = sk.kv4_attention(cfg, cache, q, torch.tensor([70, 70], dtype=torch.int32).cuda(), 0.1, ws)
        assert ws.status() == (1, 1)
        assert torch.allclose(o, full[0], atol=1e-5) and torch.allclose(lse, full[1], atol=1e-5)
    cache.page_table.copy_(table)
    for f in ([0, 100], [0, -1]):
        sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), torch.tensor(f, dtype=torch.int32).cuda(), ws)
        assert ws.status() == (1, 1), f
    o, lse = sk.kv4_attention(cfg, cache, q, torch.tensor([129, -3], dtype=torch.int32).cuda(), 0.1, ws)
    code, _ = ws.status()   # lengths past the table and below zero count as its end and as none
    assert code == 1 and not o[1].any() and lse[1].item() == -INF


def check_attention(out, lse, ref, what=""):
    """A weight enters the product to 2^-16 of itself and an exponential errs by 2^-22; a logit by a
    few 2^-22 of the products it is summed from.  An output moves by at most twice that times the
    weighted mean of |z| + 15 |s|."""
    o, l, bound, logit = ref
    dx = 2.0 ** -19 * logit + 2.0 ** -21
    compare(out.double().cpu().numpy(), o, (2.0 ** -16 + 2 * dx[..., None]) * bound + 1e-37, what + "out")
    compare(lse.double().cpu().numpy(), l, dx + 2.0 ** -21 * np.abs(np.where(np.isfinite(l), l, 0)) + 2.0 ** -16, what + "lse")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,n_q,lens", [
    (1, 1, 1, [1]), (4, 1, 1, [0, 5]), (32, 8, 1, [33, 1000]), (28, 4, 1, [64, 63, 65, 1]), (8, 1, 1, [2000]),
    (8, 2, 2, [100, 1, 0]), (7, 1, 3, [40, 2]), (6, 2, 5, [4, 300, 5]), (8, 8, 9, [77]), (16, 2, 64, [70, 64, 10]),
    (5, 5, 1, [16, 15, 17, 31, 32, 47, 48, 49, 96])])
def test_kv4_attention(sk, dtype, hq, hkv, n_q, lens):
    B, mp = len(lens), max(1, -(-max(lens) // 64))
    cfg, cache, ws = kv_cache(sk, B, hkv, mp, n_q, hq, seed=hq + n_q)
    k, v = kv_rows(dtype, B, max(1, max(lens)), hkv, 4)
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"), ws,
                  n_valid=torch.tensor(lens, dtype=torch.int32).cuda())
    # behind the last token of each sequence the pages hold NaN scales: none may show
    nan = torch.tensor([0xFF, 0x7F], dtype=torch.uint8)
    pages, table = cache.pages.cpu(), cache.page_table.cpu()
    for b, n in enumerate(lens):
        for t in range(n, mp * 64):
            tile = pages[table[b, t // 64], :, t % 64 // 16 * 2304:][:, :2304]
            for gr in range(2):
                for is_v in range(2):
                    at = kv4.param_byte(t % 16, gr, is_v)
                    tile[:, at:at + 4] = nan.repeat(2)
    cache.pages.copy_(pages)
    q = torch.randn(B, n_q, hq, 128, generator=gen(8)).to(DT[dtype])
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.11, ws)
    assert ws.status() == (0, 0)
    check_attention(out, lse, kv4.attention(q.double().numpy(), pages.numpy(), table.numpy(), lens, 0.11))
    # the same bits again, into given buffers, and with a larger workspace
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws2 = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=64)
    sk.kv4_attention(cfg, cache, q.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.11, ws2, out=o2, lse=l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def fill_cache(sk, cfg, cache, ws, lens, seed, dtype="bf16"):
    k, v = kv_rows(dtype, len(lens), max(1, max(lens)), cfg.n_kv_heads, seed)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), torch.zeros_like(n), ws, n_valid=n)
    return n


@pytest.mark.parametrize("hq,hkv,n_q,lens", [
    # more groups than CTAs: a CTA's share crosses groups, and there are more than 32 sequences
    (8, 4, 1, [(37 * i) % 190 for i in range(70)]),
    # groups for every CTA, one of them far longer than the rest
    (8, 8, 1, [20000] + [5, 0, 64] * 5), (4, 2, 4, [9000, 1, 700, 33]),
    # one group over all CTAs
    (3, 1, 1, [30000])])
def test_kv4_attention_shares(sk, hq, hkv, n_q, lens):
    B = len(lens)
    cfg, cache, ws = kv_cache(sk, B, hkv, max(1, -(-max(lens) // 64)), n_q, hq, seed=3)
    n = fill_cache(sk, cfg, cache, ws, lens, 5)
    q = torch.randn(B, n_q, hq, 128, generator=gen(9)).bfloat16()
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), n, 0.0884, ws)
    assert ws.status() == (0, 0)
    check_attention(out, lse, kv4.attention(q.double().numpy(), cache.pages.cpu().numpy(), cache.page_table.cpu().numpy(), lens, 0.0884))


def test_kv4_calls_of_different_sizes_take_turns_on_a_workspace(sk):
    """A workspace for 64 query tokens and four sequences serves calls of other batches and
    numbers of query tokens in between."""
    cfg4, c4, ws = kv_cache(sk, 4, 2, 12, 64, 16)
    n4 = fill_cache(sk, cfg4, c4, ws, [700, 64, 1, 300], 1)
    cfg1, c1, _ = kv_cache(sk, 1, 2, 12, 1, 16, seed=1)
    n1 = fill_cache(sk, cfg1, c1, ws, [750], 2)
    calls = []
    for cfg, c, n, n_q in ((cfg4, c4, n4, 64), (cfg1, c1, n1, 1), (cfg4, c4, n4, 2), (cfg1, c1, n1, 7)):
        q = torch.randn(cfg.batch, n_q, 16, 128, generator=gen(n_q)).bfloat16().cuda()
        own = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q)
        calls.append((cfg, c, q, n, sk.kv4_attention(cfg, c, q, n, 0.1, own)))
    for _ in range(2):
        for cfg, c, q, n, want in calls:
            got = sk.kv4_attention(cfg, c, q, n, 0.1, ws)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ws.status() == (0, 0)


def test_kv4_two_streams_at_once(sk):
    """Two calls side by side on streams of their own, each with its own workspace."""
    cfg, cache, ws = kv_cache(sk, 2, 2, 80, 1, 8)
    n = fill_cache(sk, cfg, cache, ws, [5000, 3000], 1)
    q = [torch.randn(2, 1, 8, 128, generator=gen(i)).bfloat16().cuda() for i in range(2)]
    want = [sk.kv4_attention(cfg, cache, x, n, 0.1, ws) for x in q]
    wss = [sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(sk.kv4_attention(cfg, cache, q[i], n, 0.1, wss[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_kv4_short_waits_time_out_and_leave_the_gpu_usable(sk):
    """With waits that give up at once the call reports the time-out (or is right, if every
    copy had landed), and the next call is right."""
    cfg, cache, ws = kv_cache(sk, 1, 2, 200, 1, 8)
    n = fill_cache(sk, cfg, cache, ws, [12000], 1)
    q = torch.randn(1, 1, 8, 128, generator=gen(1)).bfloat16().cuda()
    want = sk.kv4_attention(cfg, cache, q, n, 0.1, ws)
    assert ws.status() == (0, 0)
    short = sk.Config(1, 8, 2, 0, 0, 64, flags=sk.sekv.FLAG_SHORT_WAITS)
    got = sk.kv4_attention(short, cache, q, n, 0.1, ws)
    code, detail = ws.status()
    assert (code, detail) == (2, 4) or (code == 0 and torch.equal(got[0], want[0]))
    again = sk.kv4_attention(cfg, cache, q, n, 0.1, ws)
    assert ws.status() == (0, 0)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_kv4_attention_non_finite_queries(sk):
    """A NaN or an infinity in one head's query makes that head NaN and no other."""
    cfg, cache, ws = kv_cache(sk, 1, 1, 2, 2, 4)
    n = fill_cache(sk, cfg, cache, ws, [100], 3)
    q = torch.randn(1, 2, 4, 128, generator=gen(2)).bfloat16()
    clean = sk.kv4_attention(cfg, cache, q.cuda(), n, 0.1, ws)
    q[0, 0, 1, 77], q[0, 1, 2, 3], q[0, 1, 3, 64] = math.nan, INF, -INF
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), n, 0.1, ws)
    bad = torch.zeros(1, 2, 4, dtype=torch.bool, device="cuda")
    bad[0, 0, 1] = bad[0, 1, 2] = bad[0, 1, 3] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], clean[0][~bad])


@pytest.mark.parametrize("size", [1e-30, 1e4, 1e30])
def test_kv4_attention_values_of_any_size(sk, size):
    """Values far outside fp16's range, keys with a large common offset."""
    cfg, cache, ws = kv_cache(sk, 1, 1, 3, 1, 4)
    k, v = kv_rows("bf16", 1, 150, 1, 5)
    k, v = (k + 50).bfloat16(), (v.float() * size).bfloat16()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), zero, ws)
    q = torch.randn(1, 1, 4, 128, generator=gen(2)).bfloat16()
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), zero + 150, 0.088, ws)
    check_attention(out, lse, kv4.attention(q.double().numpy(), cache.pages.cpu().numpy(), cache.page_table.cpu().numpy(), [150], 0.088))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("at", [6, 71])
def test_kv4_attention_query_outlier(sk, dtype, at):
    """One dimension (of an even and of an odd place) far larger than the others, where the keys
    are small: the other dimensions still count."""
    cfg, cache, ws = kv_cache(sk, 1, 1, 3, 1, 4)
    k = torch.randint(0, 16, (1, 150, 1, 128), generator=gen(1)).float()
    k[..., 0], k[..., 1], k[..., 64], k[..., 65], k[..., at] = 0, 15, 0, 15, 1
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, k.to(DT[dtype]).cuda(), kv_rows(dtype, 1, 150, 1, 5)[1].cuda(), zero, ws)
    q = torch.randn(1, 1, 4, 128, generator=gen(2))
    q[..., at] = 64
    q = q.to(DT[dtype])
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), zero + 150, 0.088, ws)
    check_attention(out, lse, kv4.attention(q.double().numpy(), cache.pages.cpu().numpy(), cache.page_table.cpu().numpy(), [150], 0.088))


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("T", [31, 700, 9000])
def test_kv4_attention_every_other_token(sk, odd, T):
    """Only the even or only the odd tokens have weight."""
    cfg, cache, ws = kv_cache(sk, 1, 1, -(-T // 64), 1, 2)
    k, v = kv_rows("bf16", 1, T, 1, 5)
    q = torch.randn(1, 1, 2, 128, generator=gen(2)).bfloat16()
    u = q[0, 0].float().sum(0)
    k = (0.1 * k.float() + torch.where(torch.arange(T) % 2 == odd, 1.0, -1.0).view(1, T, 1, 1) * u).bfloat16()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), zero, ws)
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), zero + T, 0.088, ws)
    check_attention(out, lse, kv4.attention(q.double().numpy(), cache.pages.cpu().numpy(), cache.page_table.cpu().numpy(), [T], 0.088))


def test_kv4_masked_row_with_nan_does_not_show(sk):
    """Draft tokens: a later token's K and V hold NaN; the queries before it stay clean."""
    cfg, cache, ws = kv_cache(sk, 1, 1, 1, 3, 2)
    k, v = kv_rows("bf16", 1, 20, 1, 6)
    v[0, 19, 0, 3] = k[0, 19, 0, 90] = math.nan
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), zero, ws)
    q = torch.randn(1, 3, 2, 128, generator=gen(2)).bfloat16()
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), zero + 20, 0.1, ws)
    ref = kv4.attention(q[:, :2].double().numpy(), cache.pages.cpu().numpy(), cache.page_table.cpu().numpy(), [19], 0.1)
    check_attention(out[:, :2], lse[:, :2], ref)
    assert torch.isnan(out[:, 2]).all() and torch.isnan(lse[:, 2]).all()


def test_kv4_long_context_and_far_pages(sk):
    """A context of many chunks per CTA, whose last page lies beyond 2^31 bytes in the pool."""
    T, H = 40000, 2
    mp = -(-T // 64)
    cfg = sk.Config(1, 8, H, 0, 0, 64)
    n = (1 << 31) // (H * 9216) + 700
    pages = torch.empty(n, H, 9216, dtype=torch.uint8, device="cuda")
    table = (n - 1 - torch.randperm(mp, generator=gen(0))).int().view(1, mp).cuda()
    cache = sk.Kv4Cache(cfg, pages, table)
    ws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    k, v = kv_rows("bf16", 1, T, H, 7)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), zero, ws)
    q = torch.randn(1, 1, 8, 128, generator=gen(1)).bfloat16()
    out, lse = sk.kv4_attention(cfg, cache, q.cuda(), zero + T, 0.088, ws)
    assert ws.status() == (0, 0)
    # the oracle's pages: only those in use
    small = pages[table[0].long()].cpu().numpy()
    check_attention(out, lse, kv4.attention(q.double().numpy(), small, np.arange(mp)[None], [T], 0.088))


def test_kv4_workspace_and_shape_refusals(sk):
    cfg, cache, ws = kv_cache(sk, 2, 2, 2, 1, 16)
    q = torch.zeros(2, 9, 16, 128, dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(sk.SekvError) as e:   # a workspace made for one query token
        sk.kv4_attention(cfg, cache, q.repeat(1, 7, 1, 1), lens, 1.0, ws)
    assert e.value.status == -2
    with pytest.raises(sk.SekvError) as e:
        sk.kv4_attention(cfg, cache, torch.zeros(2, 65, 16, 128, dtype=torch.bfloat16, device="cuda"), lens, 1.0, ws)
    assert e.value.status == -5
    with pytest.raises(TypeError):
        sk.kv4_attention(cfg, cache, q.float(), lens, 1.0, ws)
    with pytest.raises(ValueError):
        sk.kv4_attention(cfg, cache, q[:1], lens, 1.0, ws)
    with pytest.raises(ValueError):
        sk.kv4_attention(cfg, cache, q, lens[:1], 1.0, ws)
    with pytest.raises(ValueError):
        sk.Kv4Cache(cfg, cache.pages, cache.page_table[:, ::2])
    with pytest.raises(sk.SekvError):
        sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=65)
    with pytest.raises(ValueError):   # a workspace of another kind of call
        sk.kv4_attention(cfg, cache, q, lens, 1.0, sk.Workspace(cfg))
    k = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        sk.kv4_append(cfg, cache, k, k[:, :, :1], lens, ws)
    with pytest.raises(sk.SekvError) as e:
        sk.kv4_append(cfg, cache, torch.zeros(2 * 300, dtype=torch.bfloat16, device="cuda").as_strided((2, 1, 2, 128), (300, 300, 130, 1)), k, lens, ws)
    assert e.value.status == -1


# ------------------------------------------------------------------ streams, graphs, together
def test_operators_on_a_side_stream_and_in_a_graph(sk, ws):
    """A decode step -- rotate, append, attend, log-probabilities -- captured once and replayed
    over changing inputs gives what eager calls on another stream give."""
    B, hq, hkv, V = 2, 8, 2, 900
    cfg, cache, wsk = kv_cache(sk, B, hkv, 3, 1, hq)
    wsg = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    plan = sk.RopePlan(128, 10000.0)
    q, k, v = (torch.empty(B, 1, h, 128, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    pos = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    first, lens = pos[:, 0], torch.ones(B, dtype=torch.int32, device="cuda")
    first = torch.zeros(B, dtype=torch.int32, device="cuda")
    logits, tok = torch.empty(B, V, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")

    def step(c, w):
        qo, ko = sk.rope(plan, q, k, pos)
        sk.kv4_append(cfg, c, ko, v, first, w)
        o, lse = sk.kv4_attention(cfg, c, qo, lens, 0.0884, w)
        r = sk.token_logprobs(logits, tok, ws, n_top=3)
        return o, lse, r.logprob, r.top_ids

    eager_cache = sk.Kv4Cache(cfg, cache.pages.clone(), cache.page_table)

    def fill(t):
        g = gen(t)
        for x in (q, k, v, logits):
            x.copy_(torch.randn(x.shape, generator=g))
        pos.fill_(t); first.fill_(t); lens.fill_(t + 1); tok.fill_(t)

    fill(0)
    step(cache, wsg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache, wsg)
    side = torch.cuda.Stream()
    for t in range(100):
        fill(t)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = step(eager_cache, wsk)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b), t
    assert wsk.status() == (0, 0) and wsg.status() == (0, 0) and ws.status() == (0, 0)


def test_operators_follow_each_other_without_a_wait(sk, ws):
    """Blocks of a call may be on their way while the call before it runs: each still sees all
    that came before, and overwrites nothing that is still read."""
    B, hq, hkv, T = 2, 8, 2, 5000
    cfg = sk.Config(B, hq, hkv, 0, 0, 64)
    kws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    mp = -(-T // 64)
    x = torch.randn(B, T, hq + 2 * hkv, 128, generator=gen(1)).bfloat16().cuda()
    logits = torch.randn(B, 4000, generator=gen(2)).cuda()
    plan, zero = sk.RopePlan(128), torch.zeros(B, dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")

    def chain(wait):
        cache = sk.Kv4Cache(cfg, torch.zeros(B * mp, hkv, 9216, dtype=torch.uint8, device="cuda"),
                            torch.arange(B * mp, dtype=torch.int32, device="cuda").view(B, mp))
        qkv, got = x.clone(), []
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        calls = [lambda: sk.rope(plan, q, k, pos, q_out=q, k_out=k),
                 lambda: sk.kv4_append(cfg, cache, k, v, zero, kws),
                 lambda: got.extend(sk.kv4_attention(cfg, cache, q[:, -1:].contiguous(), zero + T, 0.0884, kws)),
                 lambda: got.extend(sk.kv4_read(cfg, cache, zero, T, kws)),
                 lambda: k.copy_(got[-2].transpose(1, 2)),
                 lambda: sk.kv4_append(cfg, cache, v, k, zero, kws),
                 lambda: got.extend(sk.kv4_attention(cfg, cache, q[:, -1:].contiguous(), zero + T, 0.0884, kws)),
                 lambda: got.append(sk.token_logprobs(logits, zero.long(), ws, n_top=4).top_logprobs)]
        for _ in range(3):
            for f in calls:
                f()
                if wait:
                    torch.cuda.synchronize()
        return got

    want = chain(True)
    for _ in range(5):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)
    assert kws.status() == (0, 0) and ws.status() == (0, 0)


def test_prefill_through_the_operators_into_the_span_cache(sk):
    """Logits to surprisal, projection to rotated keys, both into the 4-bit cache and
    the span build: the calls a program makes in order, each on the other's outputs."""
    import oracle
    T, hq, hkv, V = 600, 4, 2, 300
    g = gen(11)
    cfg = sk.Config(1, hq, hkv, 4, 16, 256, 16, 2, 64, 6.0)
    qkv = torch.randn(1, T, hq + 2 * hkv, 128, generator=g).bfloat16().cuda()
    logits = (torch.randn(1, T, V, generator=g) * 2).bfloat16().cuda()
    tok = torch.randint(0, V, (1, T), generator=g).cuda()
    W = (torch.randn(hkv, 64, 128, generator=g) / 128 ** 0.5).cuda()
    gates = torch.rand(1, hkv, 2, 256, 16, generator=g).cuda()
    bws = sk.Workspace(cfg, which=sk.sekv.SEKV_CALL_BUILD, ctx_len=T)
    H = sk.surprisal(logits, tok, bws)
    compare(H.double().cpu().numpy(), tokens.surprisal(logits.double().cpu().numpy(), tok.cpu().numpy()), 2.0 ** -22 * 80, "H")
    K = torch.empty(1, hkv, T, 128, dtype=torch.bfloat16, device="cuda")
    plan = sk.RopePlan(128, 500000.0, scaling="banded", factor=8.0)
    q, _ = sk.rope(plan, qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], torch.arange(T, dtype=torch.int32, device="cuda"), k_out=K.transpose(1, 2))
    f, m = tokens.rope_frequencies(128, 500000.0, "banded", 8.0)
    pos = torch.arange(T)[None]
    check_rope(K.transpose(1, 2), qkv[:, :, hq:hq + hkv].cpu(), pos, f, m, False, "bf16")
    mp = -(-T // 64)
    cache = sk.Kv4Cache(cfg, sk.alloc_kv4_pages(cfg, mp), torch.arange(mp, dtype=torch.int32, device="cuda")[None].contiguous())
    ws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk.kv4_append(cfg, cache, K.transpose(1, 2), qkv[:, :, hq + hkv:], zero, ws)
    last = q[:, -1:].contiguous()
    o, lse = sk.kv4_attention(cfg, cache, last, zero + T, 0.0884, ws)
    check_attention(o, lse, kv4.attention(last.double().cpu().numpy(), cache.pages.cpu().numpy(), cache.page_table.cpu().numpy(), [T], 0.0884))
    # the span build over what the 4-bit cache holds, cut at the computed surprisal
    Kd, Vd = sk.kv4_read(cfg, cache, zero, T, ws)
    out = sk.alloc_cache(cfg, 16 << 20)
    sk.build_spans(cfg, Kd, Vd, H, W, gates, out, bws)
    assert bws.status() == (0, 0) and ws.status() == (0, 0)
    starts, _ = oracle.segment(H[0].cpu().numpy(), 4, 16, 6.0, 2, 64)
    assert int(out["n_spans"][0]) == len(starts)
    dws = sk.Workspace(cfg)
    od, lsed, _, _ = sk.decode_step(cfg, sk.LayerCache(out), last[:, 0].contiguous(), W, torch.full((hq,), -100.0, device="cuda"), 0.0884, dws)
    assert dws.status() == (0, 0) and torch.isfinite(od).all() and torch.isfinite(lsed).all()
