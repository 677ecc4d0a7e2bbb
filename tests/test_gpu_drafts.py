"""GPU parity of tree attention over the 4-bit cache and of keeping a branch against their fp64 oracles, and a
step with drafted tokens."""
import math

import numpy as np
import pytest
import torch

from oracle import kv4
from test_gpu_operators import DT, INF, check_attention, gen, kv_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sk():
    from decode_attention_span_gb300 import build
    build.build()
    import decode_attention_span_gb300 as sk
    return sk


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def wide_pages(B, hq, hkv, n_q):
    """Pages of a table for which the kernel of many columns is taken, if it ever is."""
    g = hq // hkv
    gain = 1.84 * -(-n_q // (8 // g)) - 9.1 * -(-n_q * g // 128)
    return 1 + int(18000 / (gain * B * hkv)) if gain > 0 else 0


def cache_of(sk, B, hq, hkv, n_q, tokens, wide, seed=0):
    """A cache whose table has the pages of `tokens`, and, for the kernel of many columns, enough that
    no token reaches."""
    used = max(1, -(-tokens // 64))
    mp = max(used, wide_pages(B, hq, hkv, n_q)) if wide else used
    cfg = sk.Config(B, hq, hkv, 0, 0, 64)
    pages = torch.zeros(B * used + 2, hkv, 9216, dtype=torch.uint8, device="cuda")
    table = torch.zeros(B, mp, dtype=torch.int32)
    table[:, :used] = torch.randperm(B * used + 2, generator=gen(seed))[: B * used].view(B, used)
    ws = sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=n_q)
    return cfg, sk.Kv4Cache(cfg, pages, table.cuda()), ws


def trees(B, n, seed):
    rng, out = np.random.default_rng(seed), []
    for _ in range(B):
        m = []
        for i in range(n):
            up = int(rng.integers(max(-1, i - 9), i))
            m.append((m[up] if up >= 0 else 0) | 1 << i)
        out.append(m)
    return out


def masks(t):
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in m] for m in t], dtype=torch.int64).cuda()


def put(sk, cfg, cache, ws, k, v, lens):
    sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), i32([0] * cfg.batch), ws, n_valid=i32(lens))


def nan_behind(cache, lens, used):
    """NaN scales behind the last token of each sequence: none may show."""
    pages, table = cache.pages.cpu(), cache.page_table.cpu()
    nan = torch.tensor([0xFF, 0x7F, 0xFF, 0x7F], dtype=torch.uint8)
    for b, n in enumerate(lens):
        for t in range(n, used * 64):
            tile = pages[table[b, t // 64], :, t % 64 // 16 * 2304:][:, :2304]
            for g in range(2):
                for is_v in range(2):
                    at = kv4.param_byte(t % 16, g, is_v)
                    tile[:, at:at + 4] = nan
    cache.pages.copy_(pages)


def oracle_of(q, cache, first, tree, scale, used):
    return kv4.tree_attention(q.double().numpy(), cache.pages.cpu().numpy(), cache.page_table.cpu().numpy()[:, :used], first, tree, scale)


# ------------------------------------------------------------------ trees
CASES = [(8, 1, 1, [0]), (1, 1, 1, [64]), (2, 1, 2, [70, 3]), (4, 1, 3, [5, 0]), (32, 8, 6, [33]), (28, 4, 5, [64, 63, 1]), (8, 2, 16, [48, 112]), (7, 1, 64, [300]),
         (8, 1, 64, [0, 1, 700]), (16, 2, 64, [64, 10]), (6, 2, 61, [191]), (8, 8, 33, [77, 5])]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hkv,n_q,first", CASES)
def test_tree_attention(sk, dtype, wide, hq, hkv, n_q, first):
    if wide and not wide_pages(1, hq, hkv, n_q):
        pytest.skip("never taken by the kernel of many columns")
    B, lens = len(first), [f + n_q for f in first]
    cfg, cache, ws = cache_of(sk, B, hq, hkv, n_q, max(lens), wide, hq + n_q)
    k, v = kv_rows(dtype, B, max(lens), hkv, 4)
    put(sk, cfg, cache, ws, k, v, lens)
    used = -(-max(lens) // 64)
    nan_behind(cache, lens, used)
    q = torch.randn(B, n_q, hq, 128, generator=gen(8)).to(DT[dtype])
    tree = trees(B, n_q, 3)
    out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32(first), masks(tree), 0.11, ws)
    assert sk.last_launch_count() == (2 if wide else 1)  # its pieces are joined by a second one
    assert ws.status() == (0, 0)
    check_attention(out, lse, oracle_of(q, cache, first, tree, 0.11, used))
    # the same bits again, into given buffers
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    sk.kv4_tree_attention(cfg, cache, q.cuda(), i32(first), masks(tree), 0.11, ws, out=o2, lse=l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_tree_that_is_a_chain_gives_the_same_bits(sk):
    cfg, cache, ws = cache_of(sk, 2, 8, 2, 5, 300, False)
    k, v = kv_rows("bf16", 2, 300, 2, 4)
    put(sk, cfg, cache, ws, k, v, [300, 180])
    q = torch.randn(2, 5, 8, 128, generator=gen(1)).bfloat16().cuda()
    want = sk.kv4_attention(cfg, cache, q, i32([300, 180]), 0.09, ws)
    chain = torch.tensor([(1 << (i + 1)) - 1 for i in range(5)], dtype=torch.int64).cuda()  # one for both
    got = sk.kv4_tree_attention(cfg, cache, q, i32([295, 175]), chain, 0.09, ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # bits from n_q on count for nothing
    got = sk.kv4_tree_attention(cfg, cache, q, i32([295, 175]), chain | (-1 << 5), 0.09, ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("wide", [False, True])
def test_tree_masks_of_any_kind(sk, wide):
    """Masks that leave nothing, that leave everything, and that are no tree; no prefix in one sequence."""
    cfg, cache, ws = cache_of(sk, 2, 8, 1, 64, 200, wide)
    k, v = kv_rows("bf16", 2, 200, 1, 5)
    put(sk, cfg, cache, ws, k, v, [64, 164])
    q = torch.randn(2, 64, 8, 128, generator=gen(2)).bfloat16()
    full = (1 << 64) - 1
    tree = [[0 if i % 3 == 0 else full if i % 3 == 1 else (0x5555 << i) & full for i in range(64)] for _ in range(2)]
    out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32([0, 100]), masks(tree), 0.1, ws)
    assert ws.status() == (0, 0)
    check_attention(out, lse, oracle_of(q, cache, [0, 100], tree, 0.1, 4))
    assert not out[0, ::3].any() and (lse[0, ::3] == -INF).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("side", ["k", "v"])
def test_tree_sibling_with_nan_does_not_show(sk, wide, side):
    cfg, cache, ws = cache_of(sk, 1, 8, 1, 64, 130, wide)
    k, v = kv_rows("bf16", 1, 130, 1, 6)
    (k if side == "k" else v)[0, 70, 0, 3] = math.nan  # drafted token 4
    put(sk, cfg, cache, ws, k, v, [130])
    q = torch.randn(1, 64, 8, 128, generator=gen(2)).bfloat16()
    tree = [[(1 << i) | (16 if i in (9, 40) else 0) for i in range(64)]]
    out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32([66]), masks(tree), 0.1, ws)
    see = [i in (4, 9, 40) for i in range(64)]
    hide = [i for i in range(64) if not see[i]]
    ref = oracle_of(q, cache, [66], tree, 0.1, 3)
    check_attention(out[:, hide], lse[:, hide], [r[:, hide] for r in ref])
    at = torch.tensor([i for i in range(64) if see[i]]).cuda()
    if side == "k":
        assert torch.isnan(out[0, at]).all() and torch.isnan(lse[0, at]).all()
    else:  # a group of dimensions
        assert torch.isnan(out[0, at, :, :64]).all() and not torch.isnan(out[0, at, :, 64:]).any() and not torch.isnan(lse).any()


def rising(T, hkv, n_q, g, step, seed):
    """Keys whose logits move by `step` of log2 each 32 tokens for every query, and the queries."""
    k, v = kv_rows("bf16", 1, T, hkv, seed)
    u = torch.zeros(128)
    u[:8] = 1.0
    q = 0.2 * torch.randn(1, n_q, hkv * g, 128, generator=gen(seed + 1))
    q[..., :8] = 1.0
    k = 0.2 * k.float()
    k[..., :8] = (torch.arange(T) // 32 * step * math.log(2) / 8).view(1, T, 1, 1)
    return k.bfloat16(), v, q.bfloat16()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("step", [3.0, 9.0, 20.0, -9.0])
def test_tree_attention_of_rising_and_falling_logits(sk, wide, step):
    """Each half page outweighs all before it, or is outweighed: the references and the values move at every
    step, while products with the weights before are still under way."""
    T, n_q = 3000, 64
    cfg, cache, ws = cache_of(sk, 1, 8, 1, n_q, T, wide)
    k, v, q = rising(T, 1, n_q, 8, step, 7)
    put(sk, cfg, cache, ws, k, v, [T])
    tree = trees(1, n_q, 5)
    first = i32([T - n_q])
    out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), first, masks(tree), 1.0, ws)
    check_attention(out, lse, oracle_of(q, cache, [T - n_q], tree, 1.0, -(-T // 64)))
    for _ in range(10):
        again = sk.kv4_tree_attention(cfg, cache, q.cuda(), first, masks(tree), 1.0, ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 40, 1e30])
@pytest.mark.parametrize("at", [3, 600, 1290])
def test_tree_attention_beside_a_token_of_large_scale(sk, wide, big, at):
    """One token of far larger values, without weight, or with all of it: no token takes bits from the others by
    the size of its values alone."""
    T, n_q = 1300, 64
    for weight in (-60.0, 0.0, 20.0):
        cfg, cache, ws = cache_of(sk, 1, 8, 1, n_q, T, wide)
        k, v = kv_rows("bf16", 1, T, 1, 9)
        v[0, at] = (v[0, at].float() * big).bfloat16()
        q = torch.randn(1, n_q, 8, 128, generator=gen(3))
        q[..., 0] = 8.0
        k[..., 0] = 0
        k[0, at, 0, 0] = weight
        q = q.bfloat16()
        put(sk, cfg, cache, ws, k, v, [T])
        tree = [[(1 << (i + 1)) - 1 for i in range(n_q)]]
        out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32([T - n_q]), masks(tree), 0.1, ws)
        check_attention(out, lse, oracle_of(q, cache, [T - n_q], tree, 0.1, -(-T // 64)), "%g " % weight)


@pytest.mark.parametrize("ks,vs", [(1e-30, 1.0), (1.0, 1e-30), (1e-36, 1e30), (1e18, 1e-18), (1.0, 0.0)])
def test_tree_attention_of_any_scale(sk, ks, vs):
    """Keys and values of any size, groups of one token far apart, and constant groups (a scale of 0)."""
    T, n_q = 700, 64
    cfg, cache, ws = cache_of(sk, 1, 8, 1, n_q, T, True)
    k, v = (x.float() for x in kv_rows("bf16", 1, T, 1, 11))
    k, v = (k * ks).bfloat16(), (v * vs).bfloat16()
    v[0, ::7, 0, 64:] = (v[0, ::7, 0, 64:].float() * 2.0 ** -30).bfloat16()
    v[0, 5::11] = vs
    put(sk, cfg, cache, ws, k, v, [T])
    q = torch.randn(1, n_q, 8, 128, generator=gen(3)).bfloat16()
    tree, scale = trees(1, n_q, 1), min(0.1 / ks, 1e37)
    out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32([T - n_q]), masks(tree), scale, ws)
    check_attention(out, lse, oracle_of(q, cache, [T - n_q], tree, float(np.float32(scale)), -(-T // 64)))


def test_tree_attention_queries_of_any_size_and_not_finite(sk):
    T, n_q = 200, 64
    cfg, cache, ws = cache_of(sk, 1, 8, 1, n_q, T, True)
    k, v = kv_rows("bf16", 1, T, 1, 2)
    put(sk, cfg, cache, ws, k, v, [T])
    q = torch.randn(1, n_q, 8, 128, generator=gen(5))
    q[0, 3] *= 1e-30
    q[0, 4, 1, 6], q[0, 4, 2, 71] = 64.0, 300.0
    q[0, 5, 0, 100], q[0, 6, 1, 0], q[0, 7, 2, 127] = math.nan, INF, -INF
    q = q.bfloat16()
    tree = trees(1, n_q, 1)
    out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32([T - n_q]), masks(tree), 0.1, ws)
    bad = torch.zeros(1, n_q, 8, dtype=torch.bool)
    bad[0, 5, 0] = bad[0, 6, 1] = bad[0, 7, 2] = True
    assert torch.isnan(out[bad.cuda()]).all() and torch.isnan(lse[bad.cuda()]).all()
    clean = torch.where(bad[..., None], 0.0, q.float())
    ref = oracle_of(clean, cache, [T - n_q], tree, 0.1, 4)
    good = ~bad.numpy()
    check_attention(out[~bad.cuda()], lse[~bad.cuda()], [r[good] for r in ref])


@pytest.mark.parametrize("hq,hkv,n_q,first", [
    (8, 1, 64, [(53 * i) % 190 for i in range(90)]),     # more groups than are ever cut
    (8, 2, 64, [20000, 5, 0, 3000]),                     # one far longer than the rest
    (4, 1, 64, [9000])])
def test_tree_attention_shares(sk, hq, hkv, n_q, first):
    B, lens = len(first), [f + n_q for f in first]
    cfg, cache, ws = cache_of(sk, B, hq, hkv, n_q, max(lens), True)
    for b0 in range(0, max(lens), 4096):  # in parts
        n = min(4096, max(lens) - b0)
        k, v = kv_rows("bf16", B, n, hkv, 4 + b0)
        sk.kv4_append(cfg, cache, k.cuda(), v.cuda(), i32([b0] * B), ws, n_valid=i32([min(max(x - b0, 0), n) for x in lens]))
    q = torch.randn(B, n_q, hq, 128, generator=gen(8)).bfloat16()
    tree = trees(B, n_q, 3)
    out, lse = sk.kv4_tree_attention(cfg, cache, q.cuda(), i32(first), masks(tree), 0.1, ws)
    assert ws.status() == (0, 0)
    some = [b for b in range(B) if b % 17 == 0 or lens[b] > 2000][:6]
    for b in some:  # a few of the drafted tokens
        rows = [0, 17, 40, 63]
        check_attention(out[b, rows][None], lse[b, rows][None], dense(q, cache, b, first, tree, rows))


def dense(q, cache, b, first, tree, rows):
    """The oracle's form for a long context and a few of its drafted tokens."""
    hq, hkv = q.shape[2], cache.n_kv_heads
    pages, table = cache.pages.cpu().numpy(), cache.page_table.cpu().numpy()
    shape = (1, len(rows), hq)
    out, lse, bound, logit = np.zeros((*shape, 128)), np.zeros(shape), np.zeros((*shape, 128)), np.zeros(shape)
    for c in range(hkv):
        K, V, ka, va = kv4.get(pages, table, b, c, first[b] + q.shape[1])
        for n, i in enumerate(rows):
            seen = list(range(first[b])) + [first[b] + j for j in range(q.shape[1]) if tree[b][i] >> j & 1]
            for h in range(c * (hq // hkv), (c + 1) * (hq // hkv)):
                x = K[seen] @ q[b, i, h].double().numpy() * 0.1
                e = np.exp(x - x.max())
                p = e / e.sum()
                out[0, n, h], lse[0, n, h] = p @ V[seen], x.max() + math.log(e.sum())
                bound[0, n, h], logit[0, n, h] = np.repeat(p @ va[seen], 64), 0.1 * np.abs(q[b, i, h].double().numpy()).sum() * ka[seen].max()
    return out, lse, bound, logit


@pytest.mark.parametrize("wide", [False, True])
def test_tree_bad_pages_and_positions_are_flagged(sk, wide):
    cfg, cache, ws = cache_of(sk, 2, 8, 1, 64, 200, wide)
    k, v = kv_rows("bf16", 2, 200, 1, 5)
    put(sk, cfg, cache, ws, k, v, [200, 200])
    q = torch.randn(2, 64, 8, 128, generator=gen(1)).bfloat16().cuda()
    t = masks(trees(2, 64, 2))
    full = sk.kv4_tree_attention(cfg, cache, q, i32([136, 136]), t, 0.1, ws)
    table = cache.page_table.clone()
    for bad in (-1, cache.pages.shape[0], 1 << 30):
        cache.page_table.copy_(table)
        cache.page_table[1, 1] = bad
        out, lse = sk.kv4_tree_attention(cfg, cache, q, i32([136, 136]), t, 0.1, ws)
        assert ws.status() == (1, 1)
        assert torch.equal(out[0], full[0][0]) and torch.isfinite(out).all() and not torch.equal(out[1], full[0][1])
    cache.page_table.copy_(table)
    out, lse = sk.kv4_tree_attention(cfg, cache, q, i32([136, -1]), t, 0.1, ws)
    assert ws.status() == (1, 1) and torch.equal(out[0], full[0][0]) and not out[1].any() and (lse[1] == -INF).all()
    for f in (cache.page_table.shape[1] * 64 - 10, 2 ** 31 - 5):  # drafted tokens past the table
        cache.page_table[1] = table[1, 0]
        out, lse = sk.kv4_tree_attention(cfg, cache, q, i32([136, f]), t, 0.1, ws)
        assert ws.status() == (1, 1) and torch.isfinite(out).all()
        # the other sequence, whose pieces may be cut elsewhere now
        check_attention(out[:1], lse[:1], oracle_of(q[:1].cpu(), cache, [136], trees(2, 64, 2)[:1], 0.1, 4))


def test_tree_workspaces_take_turns(sk):
    """A wide call leaves what the other calls' counters need zero, whatever their sizes."""
    B, hkv, n_q = 40, 8, 64
    cfg, cache, ws = cache_of(sk, B, 32, hkv, n_q, 150, False)
    k, v = kv_rows("bf16", B, 150, hkv, 4)
    put(sk, cfg, cache, ws, k, v, [150] * B)
    q = torch.randn(B, n_q, 32, 128, generator=gen(1)).bfloat16().cuda()
    want = sk.kv4_attention(cfg, cache, q, i32([150] * B), 0.1, ws)
    cfg1, cache1, _ = cache_of(sk, 1, 8, 1, n_q, 3000, True)
    k1, v1 = kv_rows("bf16", 1, 3000, 1, 4)
    put(sk, cfg1, cache1, ws, k1, v1, [3000])
    q1, t1 = torch.randn(1, n_q, 8, 128, generator=gen(2)).bfloat16().cuda(), masks(trees(1, n_q, 1))
    first = sk.kv4_tree_attention(cfg1, cache1, q1, i32([2900]), t1, 0.1, ws)
    for _ in range(3):
        got = sk.kv4_attention(cfg, cache, q, i32([150] * B), 0.1, ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        again = sk.kv4_tree_attention(cfg1, cache1, q1, i32([2900]), t1, 0.1, ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert ws.status() == (0, 0)


def test_tree_short_waits_time_out_and_leave_the_gpu_usable(sk):
    cfg, cache, ws = cache_of(sk, 1, 8, 2, 64, 5000, True)
    k, v = kv_rows("bf16", 1, 5000, 2, 4)
    put(sk, cfg, cache, ws, k, v, [5000])
    q, t = torch.randn(1, 64, 8, 128, generator=gen(1)).bfloat16().cuda(), masks(trees(1, 64, 2))
    want = sk.kv4_tree_attention(cfg, cache, q, i32([4936]), t, 0.1, ws)
    short = sk.Config(1, 8, 2, 0, 0, 64, flags=2)
    sk.kv4_tree_attention(short, cache, q, i32([4936]), t, 0.1, ws)
    assert ws.status()[0] == 2
    got = sk.kv4_tree_attention(cfg, cache, q, i32([4936]), t, 0.1, ws)
    assert ws.status() == (0, 0) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ keeping a branch
@pytest.mark.parametrize("B,hkv,first,keep,n_keep", [
    (1, 1, [0], [[0, 1, 2]], [3]), (1, 2, [61], [[1, 2, 5, 9, 40]], [5]), (3, 1, [5, 64, 200], [[3, 7, 0], [0, 2, 4], [63, 0, 0]], [2, 3, 1]),
    (2, 8, [30, 127], [list(range(1, 64)), list(range(0, 63))], None), (2, 1, [10, 20], [[9], [1]], [0, 1]),
    (2, 2, [1, 70], [[0, 2], [1, 3]], [-5, 9])])
def test_keep(sk, B, hkv, first, keep, n_keep):
    cfg, cache, ws = cache_of(sk, B, hkv, hkv, 1, max(first) + 64, False)
    pages = torch.randint(0, 256, cache.pages.shape, dtype=torch.uint8, generator=gen(3))
    cache.pages.copy_(pages)
    sk.kv4_keep(cfg, cache, i32(first), i32(keep), None if n_keep is None else i32(n_keep), ws)
    assert ws.status() == (0, 0)
    want = pages.numpy().copy()
    for b in range(B):
        n = len(keep[b]) if n_keep is None else max(0, min(n_keep[b], len(keep[b])))
        for c in range(hkv):
            kv4.keep(want, cache.page_table.cpu().numpy(), b, c, first[b], keep[b][:n])
    assert np.array_equal(cache.pages.cpu().numpy(), want)


def test_keep_refuses_lists_that_do_not_ascend(sk):
    cfg, cache, ws = cache_of(sk, 2, 1, 1, 1, 200, False)
    pages = torch.randint(0, 256, cache.pages.shape, dtype=torch.uint8, generator=gen(3))
    for bad, first in (([2, 2], 4), ([3, 1], 4), ([-1, 2], 4), ([0, 1], -3)):
        cache.pages.copy_(pages)
        sk.kv4_keep(cfg, cache, i32([100, first]), i32([[1, 5], bad]), None, ws)
        assert ws.status() == (1, 1)
        want = pages.numpy().copy()
        kv4.keep(want, cache.page_table.cpu().numpy(), 0, 0, 100, [1, 5])
        assert np.array_equal(cache.pages.cpu().numpy(), want), bad
    # a token whose page is not in the pool, or not in the table, does not move; the others do
    table = cache.page_table.clone()
    for at, far in ((1, 5), (None, 200)):
        cache.pages.copy_(pages)
        if at is not None:
            cache.page_table[1, at] = 1 << 20
        sk.kv4_keep(cfg, cache, i32([100, 60]), i32([[1, 2], [1, far]]), None, ws)
        assert ws.status() == (1, 1)
        want = pages.numpy().copy()
        kv4.keep(want, table.cpu().numpy(), 0, 0, 100, [1, 2])
        kv4.keep(want, table.cpu().numpy(), 1, 0, 60, [1])
        assert np.array_equal(cache.pages.cpu().numpy(), want), far
        cache.page_table.copy_(table)
    sk.kv4_keep(cfg, cache, i32([0, 0]), torch.zeros(2, 0, dtype=torch.int32, device="cuda"), None, ws)
    assert ws.status() == (0, 0)


# ------------------------------------------------------------------ a step with drafted tokens
@pytest.mark.parametrize("wide", [False, True])
def test_a_step_with_drafted_tokens_in_a_graph(sk, wide):
    """Append the drafted tokens, attend, score them from last states, keep a branch and read it back: eagerly on a
    side stream, and captured and replayed with other inputs."""
    B, hq, hkv, n_q, T, V, D = 2, 16, 2, 64, 300, 2000, 256
    cfg, cache, ws = cache_of(sk, B, hq, hkv, n_q, T + 64, wide)
    ws2 = sk.StatesWorkspace(B * n_q, V, D)
    k0, v0 = kv_rows("bf16", B, T, hkv, 1)
    first = i32([T, 190])
    k, v = (x.cuda() for x in kv_rows("bf16", B, n_q, hkv, 2))
    q = torch.randn(B, n_q, hq, 128, generator=gen(3)).bfloat16().cuda()
    tree, t = trees(B, n_q, 4), masks(trees(B, n_q, 4))
    x = torch.randn(B, n_q, D, generator=gen(5)).bfloat16().cuda()
    w = torch.randn(V, D, generator=gen(6)).bfloat16().cuda() / 16
    tok = torch.randint(0, V, (B, n_q), generator=gen(7)).cuda()
    kept, n_keep = i32([[0, 3, 9, 30], [1, 2, 0, 0]]), i32([4, 2])
    put(sk, cfg, cache, ws, k0, v0, [T, 190])
    fresh = cache.pages.clone()
    rk, rv = (torch.zeros(B, hkv, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")

    def step(stream=None):
        sk.kv4_append(cfg, cache, k, v, first, ws, stream=stream)
        o = sk.kv4_tree_attention(cfg, cache, q, first, t, 0.088, ws, stream=stream)
        r = sk.states_logprobs(x, w, tok, ws2, stream=stream)
        sk.kv4_keep(cfg, cache, first, kept, n_keep, ws, stream=stream)
        sk.kv4_read(cfg, cache, first, 4, ws, n_valid=n_keep, out=(rk, rv), stream=stream)
        return (*o, *r)
    want = [y.clone() for y in step()] + [rk.clone(), rv.clone(), cache.pages.clone()]
    assert ws.status() == (0, 0) and ws2.status() == (0, 0)
    cache.pages.copy_(fresh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = list(step(side))
    side.synchronize()
    for a, b in zip(got + [rk, rv, cache.pages], want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = list(step())
    for again in range(2):
        cache.pages.copy_(fresh)
        if again:
            for y in (q, x, k):
                y.neg_()
        rk.zero_(), rv.zero_()
        graph.replay()
        got = [y.clone() for y in held] + [rk.clone(), rv.clone(), cache.pages.clone()]
        cache.pages.copy_(fresh)
        now = list(step()) + [rk, rv, cache.pages]
        torch.cuda.synchronize()
        for a, b in zip(got, now):
            assert torch.equal(a, b)
    assert tree is not None and ws.status() == (0, 0)


def test_trees_on_two_streams_at_once(sk):
    sets = []
    for i in range(2):
        cfg, cache, ws = cache_of(sk, 1, 8, 1, 64, 2000, True, i)
        k, v = kv_rows("bf16", 1, 2000, 1, i)
        put(sk, cfg, cache, ws, k, v, [2000])
        q, t = torch.randn(1, 64, 8, 128, generator=gen(i)).bfloat16().cuda(), masks(trees(1, 64, i))
        want = sk.kv4_tree_attention(cfg, cache, q, i32([1936]), t, 0.1, ws)
        sets.append((cfg, cache, ws, q, t, i32([1936]), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for cfg, cache, ws, q, t, first, _, s in sets:
            got.append(sk.kv4_tree_attention(cfg, cache, q, first, t, 0.1, ws, stream=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], sets[i % 2][6][0]) and torch.equal(g[1], sets[i % 2][6][1])
