"""Host-side refusals and tables of the operators around the cache (CPU)."""
import ctypes

import numpy as np
import pytest

from turns import turns


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


def test_tensors_without_elements_may_have_no_address(libsekv):
    """What torch gives for an empty tensor is address 0."""
    import decode_attention_span_gb300 as sk
    from decode_attention_span_gb300 import rotary
    from decode_attention_span_gb300.kv4 import SekvKv4Cache
    cfg = ctypes.byref(sk.Config(1, 8, 2, 0, 0, 64).c())
    cache = ctypes.byref(SekvKv4Cache(1 << 20, 1 << 20, 4, 4))
    S = (ctypes.c_int64 * 3)(8, 8, 8)
    append = lambda n: libsekv.sekv_kv4_append(cfg, cache, 0, None, S, None, S, n, P, None, P, 0, None)  # noqa: E731
    read = lambda n: libsekv.sekv_kv4_read(cfg, cache, 0, None, None, n, P, None, P, 0, None)  # noqa: E731
    heads = lambda n, s=256: ctypes.byref(rotary.SekvHeads(0, 0, n, 0, s, 128, 0, s, 128))  # noqa: E731

    def rope(B, T, n, pos=None):
        return libsekv.sekv_rope(ctypes.byref(rotary.rope_config(64)), P, 1.0, 0, 128, B, T, pos, 0, 0, heads(n), None, 0, None)

    def logprobs(B, T):
        return libsekv.sekv_token_logprobs(None, 0, B, T, 9, 0, 9, None, 0, 0, 1.0, 0, None, None, None, None, None, P, 4096, None)

    def surprisal(B, T):
        return libsekv.sekv_surprisal(None, 0, B, T, 9, 0, 9, None, 0, 0, None, P, 4096, None)
    assert append(0) == 0 and read(0) == 0
    assert append(1) == INVALID and read(1) == INVALID
    assert rope(1, 0, 2) == 0 and rope(0, 3, 2) == 0 and rope(1, 3, 0, P) == 0 and rope(2, 0, 2) == 0
    assert rope(2, 3, 0, P) == 0                 # its strides as torch has them are 0 too
    assert rope(1, 3, 2, P) == INVALID and rope(1, 3, 2) == INVALID
    for call in (logprobs, surprisal):
        assert call(0, 3) == 0 and call(2, 0) == 0 and call(1, 2) == INVALID


@pytest.mark.parametrize("rot,base,scaling,factor", [
    (128, 500000.0, "none", 1.0), (64, 10000.0, "linear", 3.0), (128, 10000.0, "ntk", 8.0), (96, 1e6, "parts", 40.0),
    (128, 500000.0, "banded", 8.0), (512, 1e6, "none", 1.0), (2, 10000.0, "none", 1.0)])
def test_rope_table_against_fifty_digits(libsekv, rot, base, scaling, factor):
    """The table's entries against the formulas in decimals, not through fp64.  With t = ln of
    the unscaled pace, an exponent's rounding moves it by t 2^-53 of itself; the power, 2 pi, its
    quotient and the scalings' six operations by 2^-53 each; the entry is cut at 2^-63.  As
    (t + 12) e^-t is at most 12, an angle is off by 12 * 2^-53 of a radian a position, below
    2^-49."""
    from decode_attention_span_gb300 import rotary
    freqs, _ = rotary.rope_freqs(rotary.rope_config(rot, base, scaling=scaling, factor=factor))
    want = turns(rot, base, scaling, factor)
    for i, (got, w) in enumerate(zip(freqs.numpy().view(np.uint64), want)):
        off = abs(int(got) - int(w % 1 * 2 ** 64))
        off = min(off, 2 ** 64 - off) / 2.0 ** 64
        t = 2 * i / rot * np.log(base * (factor ** (rot / (rot - 2)) if scaling == "ntk" else 1))
        assert off <= (t + 12) * 2.0 ** -53 * float(w) + 2.0 ** -63, i
        assert off * 2 * np.pi <= 2.0 ** -49
