"""Frequencies of rotary embeddings to fifty digits, for tests of their table."""
import decimal
from decimal import Decimal as D

PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(rot, base, scaling="none", factor=1.0, original=8192, beta_fast=32.0, beta_slow=1.0,
          low=1.0, high=4.0):
    """Turns a position of each pair, written from the C header's formulas."""
    with decimal.localcontext() as c:
        c.prec = 60
        base, factor, d = D(base), D(factor), D(rot)
        if scaling == "ntk":
            base *= (factor.ln() * d / (d - 2)).exp()
        out = []
        for i in range(rot // 2):
            u = (-2 * i * base.ln() / d).exp()
            if scaling == "linear":
                u /= factor
            elif scaling == "parts":
                pair = lambda n: d * (original / (2 * PI * D(n))).ln() / (2 * base.ln())  # noqa: E731
                lo = max(D(0), pair(beta_fast).to_integral_value(decimal.ROUND_FLOOR))
                hi = min(d - 1, pair(beta_slow).to_integral_value(decimal.ROUND_CEILING))
                r = min(D(1), max(D(0), (i - lo) / max(hi - lo, D("0.001"))))
                u = (1 - r) * u + r * u / factor
            elif scaling == "banded":
                s = min(D(1), max(D(0), (original * u / (2 * PI) - D(low)) / D(high - low)))
                u = (1 - s) * u / factor + s * u
            out.append(u / (2 * PI))
        return out
