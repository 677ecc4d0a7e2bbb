"""GPU parity of the operators around the cache at the places where they can go wrong, against
their fp64 oracles or closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import tokens

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
