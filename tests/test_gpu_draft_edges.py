"""GPU: tree attention where it is easy to go wrong: waits that run out, long sums, workspaces."""
import time

import pytest
import torch

from test_gpu_drafts import cache_of, i32, masks, put, trees
from test_gpu_operators import gen, kv_rows

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
