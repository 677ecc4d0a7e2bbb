"""GPU: tree attention where it is easy to go wrong: waits that run out, long sums, workspaces."""
import math
import time

import numpy as np
import pytest
import torch

from oracle import kv4
from test_gpu_drafts import cache_of, i32, masks, oracle_of, put, rising, trees
from test_gpu_operators import check_attention, gen, kv_rows
from test_gpu_states import check_states

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sk():
    from decode_attention_span_gb300 import build
    build.build()
    import decode_attention_span_gb300 as sk
    return sk


@pytest.mark.parametrize("pages", range(1, 14))
def test_a_tree_that_gives_up_ends_at_once(sk, pages):
    """Of an item's pages only those are waited for at the end whose copies were issued: 32 pieces of `pages` pages
    each, of which waits that run out at once leave most untouched."""
    T = 2048 * pages - 5
    cfg, cache, ws = cache_of(sk, 1, 8, 2, 64, T, True)
    k, v = kv_rows("bf16", 1, T, 2, 4)
    put(sk, cfg, cache, ws, k, v, [T])
    q, t, first = torch.randn(1, 64, 8, 128, generator=gen(1)).bfloat16().cuda(), masks(trees(1, 64, 2)), i32([T - 64])
    want = sk.kv4_tree_attention(cfg, cache, q, first, t, 0.1, ws)
    assert ws.status() == (0, 0)
    short = sk.Config(1, 8, 2, 0, 0, 64, flags=2)
    t0 = time.monotonic()
    for _ in range(5):
        sk.kv4_tree_attention(short, cache, q, first, t, 0.1, ws)
    assert ws.status()[0] == 2
    assert time.monotonic() - t0 < 1.0
    got = sk.kv4_tree_attention(cfg, cache, q, first, t, 0.1, ws)
    assert ws.status() == (0, 0) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def shared_cache(sk, B, hkv, n_q, hq, k, v):
    """B sequences that all hold the tokens k, v [1][T][hkv][128], in the same pages."""
    T = k.shape[1]
    mp = -(-T // 64)
    one = sk.Config(1, hq, hkv, 0, 0, 64)
    pages = torch.zeros(mp, hkv, 9216, dtype=torch.uint8, device="cuda")
    table = torch.randperm(mp, generator=gen(1)).to(torch.int32)[None].cuda()
    ws = sk.Workspace(one, which=sk.SEKV_CALL_KV4, ctx_len=n_q)
    cache = sk.Kv4Cache(one, pages, table)
    sk.kv4_append(one, cache, k, v, i32([0]), ws)
    values = sk.kv4_read(one, cache, i32([0]), T, ws, out=tuple(torch.empty(1, hkv, T, 128, device="cuda") for _ in "kv"))
    cfg = sk.Config(B, hq, hkv, 0, 0, 64)
    many = sk.Kv4Cache(cfg, pages, table.expand(B, mp).contiguous())
    return cfg, many, sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q), values


@pytest.mark.parametrize("kind", ["high", "low", "constant", "any"])
@pytest.mark.parametrize("B,hq,hkv,T", [
    (20, 16, 8, 24000),     # 160 groups: more than are ever cut
    (20, 16, 8, 2100),      # a flush and little more
    (1, 32, 8, 131072),     # cut into long pieces
    (3, 7, 1, 50000)])
def test_values_that_point_one_way_over_a_long_context(sk, kind, B, hq, hkv, T):
    """Logits near 0: outputs are off by at most 2^-18 of the weighted mean of a group's largest value, and twice the
    logits' error, however long the sum is."""
    n_q = 64
    g = torch.Generator(device="cuda").manual_seed(3)
    v = 1 - 0.05 * torch.rand(1, T, hkv, 128, generator=g, device="cuda")
    if kind == "low":
        v = 1 - v
    v[..., ::64] = 1.0 if kind == "low" else 0.0     # one element of a group spreads its codes
    v *= 0.5 + 0.5 * torch.rand(1, T, hkv, 1, generator=g, device="cuda")
    if kind == "constant":
        v[:] = 0.1
    if kind == "any":
        v = torch.randn(1, T, hkv, 128, generator=g, device="cuda")
    v = v.bfloat16()
    k = torch.randn(1, T, hkv, 128, generator=g, device="cuda").bfloat16()
    cfg, cache, ws, (keys, values) = shared_cache(sk, B, hkv, n_q, hq, k, v)
    q, scale = torch.randn(B, n_q, hq, 128, generator=gen(2)).bfloat16().cuda(), 0.002
    own = torch.tensor([1 << i if i < 63 else -(1 << 63) for i in range(n_q)], dtype=torch.int64).cuda()
    out, lse = sk.kv4_tree_attention(cfg, cache, q, i32([T - n_q] * B), own, scale, ws)
    assert ws.status() == (0, 0) and sk.last_launch_count() == (1 if B * hkv > 152 else 2)
    G = hq // hkv
    hidden = torch.cat([torch.zeros(n_q, T - n_q, dtype=torch.bool), ~torch.eye(n_q, dtype=torch.bool)], 1).cuda()
    for b, c in {(0, 0), (B - 1, hkv - 1)}:
        x, y, h = keys[0, c].double(), values[0, c].double(), q[b, :, c * G:c * G + G].double()
        kmax = x.abs().amax().item()  # s is at most 2 kmax / 15 (rounded up by 2^-8), |z| + 15 |s| at most 3 kmax
        dx = scale * (2.0 ** -16 * h.abs().amax(-1) * 4.1 / 15 * kmax + 2.0 ** -22 * h.abs().sum(-1) * 3 * kmax)
        p = torch.einsum("igd,td->igt", h, x) * scale
        p.masked_fill_(hidden[:, None], float("-inf"))
        want_lse = torch.logsumexp(p, -1)
        p = torch.softmax(p, -1)
        bound = p @ y.view(T, 2, 64).abs().amax(2).repeat_interleave(64, 1)
        err = (out[b, :, c * G:c * G + G].double() - p @ y).abs() / bound
        assert (err <= 2.0 ** -18 + 2 * dx[..., None]).all(), err.max().item()
        assert ((lse[b, :, c * G:c * G + G].double() - want_lse).abs() <= 2.0 ** -18 + dx + 2.0 ** -22 * want_lse).all()


@pytest.mark.parametrize("what", [3.0, 9.0, 20.0, -9.0, "early", "late", "falling"])
def test_references_and_units_move_between_flushes(sk, what):
    """160 groups of 94 pages, none cut: what was flushed follows when logits rise by `what` of log2 each 32 tokens, and
    when tokens of far larger values come early or late or all become smaller."""
    B, hq, hkv, n_q, T = 20, 16, 8, 64, 6000
    if isinstance(what, float):
        k, v, q1 = rising(T, hkv, n_q, hq // hkv, what, 7)
        scale = 1.0
    else:
        k, v = kv_rows("bf16", 1, T, hkv, 9)
        q1, scale = torch.randn(1, n_q, hq, 128, generator=gen(3)).bfloat16(), 0.02
        v = v.float()
        if what == "falling":
            v *= 2.0 ** (30 - torch.arange(T) / 100).view(1, T, 1, 1)
        else:
            v[0, 40 if what == "early" else 5000] *= 2.0 ** 40
        v = v.bfloat16()
    cfg, cache, ws, (keys, values) = shared_cache(sk, B, hkv, n_q, hq, k.cuda(), v.cuda())
    tree = trees(1, n_q, 5)
    q = q1.cuda().expand(B, n_q, hq, 128).contiguous()
    out, lse = sk.kv4_tree_attention(cfg, cache, q, i32([T - n_q] * B), masks(tree)[0].contiguous(), scale, ws)
    assert ws.status() == (0, 0) and sk.last_launch_count() == 1
    assert torch.equal(out[0], out[B - 1]) and torch.equal(lse[0], lse[7])
    pages, table = cache.pages.cpu().numpy(), cache.page_table.cpu().numpy()
    for c in (0, hkv - 1):
        K, V, ka, va = kv4.get(pages, table, 0, c, T)
        for i in (0, 31, 63):
            seen = list(range(T - n_q)) + [T - n_q + j for j in range(n_q) if tree[0][i] >> j & 1]
            for h in (2 * c, 2 * c + 1):
                x = K[seen] @ q1[0, i, h].double().numpy() * scale
                e = np.exp(x - x.max())
                p = e / e.sum()
                ref = (p @ V[seen], x.max() + math.log(e.sum()), np.repeat(p @ va[seen], 64),
                       scale * np.abs(q1[0, i, h].double().numpy()).sum() * ka[seen].max())
                check_attention(out[3, i, h][None], lse[3, i, h][None], [np.asarray(r)[None] for r in ref])


def small_ws(sk, cfg, n_q):
    """A workspace of what the calls other than a wide tree's need: the partials of eight columns for two groups of each
    CTA, and a counter for each group."""
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, 256)
    blocks = -(-n_q // (8 // (cfg.n_q_heads // cfg.n_kv_heads)))
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    ws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=1)
    ws.nbytes = 256 + up(ctas * 2 * 8 * 130 * 4) + up(cfg.batch * cfg.n_kv_heads * blocks * 4)
    ws.buf = torch.zeros(ws.nbytes, dtype=torch.uint8, device="cuda")
    return ws


@pytest.mark.parametrize("B,hq,hkv,n_q", [(1, 8, 1, 1), (3, 28, 4, 4), (1, 32, 8, 8), (2, 8, 2, 64), (1000, 8, 8, 1)])
def test_calls_without_a_wide_tree_need_small_workspaces(sk, B, hq, hkv, n_q):
    cfg, cache, _ = cache_of(sk, B, hq, hkv, 1, 100, False)
    ws = small_ws(sk, cfg, n_q)
    full = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q)
    assert full.nbytes == ws.nbytes if n_q < 9 else full.nbytes > 40 << 20
    k, v = kv_rows("bf16", B, 100, hkv, 4)
    put(sk, cfg, cache, ws, k, v, [100] * B)
    q = torch.randn(B, n_q, hq, 128, generator=gen(1)).bfloat16().cuda()
    got = sk.kv4_attention(cfg, cache, q, i32([100] * B), 0.1, ws)
    want = sk.kv4_attention(cfg, cache, q, i32([100] * B), 0.1, full)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    sk.kv4_keep(cfg, cache, i32([90] * B), i32([[0, 2]] * B), None, ws)
    sk.kv4_read(cfg, cache, i32([90] * B), 2, ws)
    tree = masks(trees(B, n_q, 1))
    if n_q == 64:
        with pytest.raises(sk.SekvError):
            sk.kv4_tree_attention(cfg, cache, q, i32([30] * B), tree, 0.1, ws)
    elif n_q < 8:
        sk.kv4_tree_attention(cfg, cache, q, i32([30] * B), tree, 0.1, ws)
    assert ws.status() == (0, 0)
    ws.nbytes -= 256
    with pytest.raises(sk.SekvError):
        sk.kv4_attention(cfg, cache, q, i32([100] * B), 0.1, ws)


def test_more_groups_than_counters_before_a_wide_tree(sk):
    """1024 x 17 x 64 groups, whose counters lie behind what a wide tree takes: both take turns on a workspace."""
    B, hkv, n_q = 1024, 17, 64
    cfg = sk.Config(B, 8 * hkv, hkv, 0, 0, 64)
    ws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q)
    pages = torch.zeros(1, hkv, 9216, dtype=torch.uint8, device="cuda")
    one = sk.Config(1, 8 * hkv, hkv, 0, 0, 64)
    cache = sk.Kv4Cache(cfg, pages, torch.zeros(B, 1, dtype=torch.int32, device="cuda"))
    k, v = kv_rows("bf16", 1, 64, hkv, 4)
    sk.kv4_append(one, sk.Kv4Cache(one, pages, torch.zeros(1, 1, dtype=torch.int32, device="cuda")), k.cuda(), v.cuda(), i32([0]), ws)
    q = torch.randn(1, n_q, 8 * hkv, 128, generator=gen(1)).bfloat16().cuda().expand(B, -1, -1, -1).contiguous()
    cfg1, cache1, _ = cache_of(sk, 1, 8, 1, n_q, 9000, True)
    k1, v1 = kv_rows("bf16", 1, 9000, 1, 4)
    put(sk, cfg1, cache1, ws, k1, v1, [9000])
    q1, t1 = torch.randn(1, n_q, 8, 128, generator=gen(2)).bfloat16().cuda(), masks(trees(1, n_q, 1))
    first = sk.kv4_tree_attention(cfg1, cache1, q1, i32([8900]), t1, 0.1, ws)
    assert sk.last_launch_count() == 2
    for _ in range(2):
        out, lse = sk.kv4_attention(cfg, cache, q, i32([64] * B), 0.1, ws)
        assert torch.equal(out[0], out[-1]) and torch.equal(lse[5], lse[-1]) and torch.isfinite(out).all()
        again = sk.kv4_tree_attention(cfg1, cache1, q1, i32([8900]), t1, 0.1, ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    check_attention(out[:1], lse[:1], kv4.attention(q[:1].double().cpu().numpy(), pages.cpu().numpy(), np.zeros((1, 1), np.int32), [64], 0.1))
    assert ws.status() == (0, 0)


@pytest.mark.parametrize("wide", [False, True])
def test_two_steps_with_drafted_tokens_against_the_oracles(sk, wide):
    """Append drafted tokens, attend, score them from last states, keep a branch, and the same again behind it: each step's
    outputs against the oracles, on the pages that the oracle's keep leaves."""
    B, hq, hkv, n_q, T, V, D = 2, 16, 2, 64, 300, 500, 128
    cfg, cache, ws = cache_of(sk, B, hq, hkv, n_q, T + 128, wide)
    states_ws = sk.StatesWorkspace(B * n_q, V, D)
    k, v = kv_rows("bf16", B, T, hkv, 1)
    lens = [T, 190]
    put(sk, cfg, cache, ws, k, v, lens)
    branches = [([0, 3, 9, 30], [1, 2]), ([5], [0, 1, 2, 3, 40])]
    used = -(-(T + 128) // 64)
    for step in range(2):
        k, v = (x.cuda() for x in kv_rows("bf16", B, n_q, hkv, 2 + step))
        q = torch.randn(B, n_q, hq, 128, generator=gen(3 + step)).bfloat16()
        tree = trees(B, n_q, 4 + step)
        sk.kv4_append(cfg, cache, k, v, i32(lens), ws)
        out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32(lens), masks(tree), 0.088, ws)
        assert sk.last_launch_count() == (2 if wide else 1)
        check_attention(out, lse, oracle_of(q, cache, lens, tree, 0.088, used))
        x, w, tok = torch.randn(B, n_q, D, generator=gen(5)).bfloat16(), torch.randn(V, D, generator=gen(6)).bfloat16() / 8, \
            torch.randint(0, V, (B, n_q), generator=gen(7 + step))
        r = sk.states_logprobs(x.cuda(), w.cuda(), tok.cuda(), states_ws)
        check_states(r, x.view(B * n_q, D), w, tok)
        kept = branches[step]
        most = max(len(b) for b in kept)
        want = cache.pages.cpu().numpy().copy()
        for b in range(B):
            for c in range(hkv):
                kv4.keep(want, cache.page_table.cpu().numpy(), b, c, lens[b], kept[b])
        sk.kv4_keep(cfg, cache, i32(lens), i32([b + [0] * (most - len(b)) for b in kept]), i32([len(b) for b in kept]), ws)
        assert np.array_equal(cache.pages.cpu().numpy(), want)
        lens = [n + len(b) for n, b in zip(lens, kept)]
    assert ws.status() == (0, 0) and states_ws.status() == (0, 0)


def test_long_items_that_give_up_end_at_once(sk):
    """The same with items of 94 pages, whose values would be flushed."""
    B, hkv, T = 20, 8, 6000
    k, v = kv_rows("bf16", 1, T, hkv, 9)
    cfg, cache, ws, _ = shared_cache(sk, B, hkv, 64, 16, k.cuda(), v.cuda())
    q, t, first = torch.randn(B, 64, 16, 128, generator=gen(1)).bfloat16().cuda(), masks(trees(B, 64, 2)), i32([T - 64] * B)
    want = sk.kv4_tree_attention(cfg, cache, q, first, t, 0.1, ws)
    short = sk.Config(B, 16, hkv, 0, 0, 64, flags=2)
    assert ws.status() == (0, 0)
    t0 = time.monotonic()
    for _ in range(5):
        sk.kv4_tree_attention(short, cache, q, first, t, 0.1, ws)
    assert ws.status()[0] == 2
    assert time.monotonic() - t0 < 1.0
    got = sk.kv4_tree_attention(cfg, cache, q, first, t, 0.1, ws)
    assert ws.status() == (0, 0) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
