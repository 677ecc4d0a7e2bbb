"""GPU: log-probabilities from last states and their gradient where it is easy to go wrong: waits that run out,
factors far apart, long sums."""
import time

import pytest
import torch

from test_gpu_states import inputs

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
