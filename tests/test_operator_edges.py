"""Host-side refusals and tables of the operators around the cache (CPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def libsekv():
    from decode_attention_span_gb300 import build, sekv
    build.build()
    return sekv.lib()


P = ctypes.c_void_p(1 << 20)   # an aligned address that no call here dereferences
INVALID = -1


def test_scales_beyond_fp32_to_the_base_two_are_refused(libsekv):
    """scale * log2(e) past fp32 would make 0 * infinity of the likeliest token's exponent."""
    import decode_attention_span_gb300 as sk
    from decode_attention_span_gb300.kv4 import SekvKv4Cache
    cfg = ctypes.byref(sk.Config(1, 8, 2, 0, 0, 64).c())
    cache = ctypes.byref(SekvKv4Cache(1 << 20, 1 << 20, 4, 4))
    logprobs = lambda scale: libsekv.sekv_token_logprobs(  # noqa: E731
        P, 0, 0, 4, 100, 0, 100, P, 0, 0, scale, 0, P, None, None, None, None, P, 4096, None)  # no rows: no launch
    attention = lambda scale: libsekv.sekv_kv4_attention(cfg, cache, 0, P, 1, P, scale, P, P, P, 0, None)  # noqa: E731
    for call in (logprobs, attention):
        for scale in (3.4e38, 2.5e38):
            assert call(scale) == INVALID
        assert call(2.0 ** 127) != INVALID
