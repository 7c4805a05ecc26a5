"""The frequencies of a rotation against their formulas in 60 decimal digits (host only).

With u = 2^-53 and a frequency w = theta^-x, x = 2 j / rot_dim:  x is exact where rot_dim is a power of two, else off
by u of itself, which moves w by |ln w| u;  pow by an ulp, 2 u;  2^64 / 2 pi by u, the product with it by u, and the
whole number that it is cut to by 2^-64 of a revolution.  A division by the factor adds u.  For bands the turns over the
context are off by another 4 u (2 pi, product, quotient), the blend m by turns / (high - low) times that and 4 u of
itself, which moves w (1 - 1 / factor) as much, and the blend of the two frequencies rounds four times.  For the ramp m
is off by 4 u."""
import math
from decimal import Decimal as D
from decimal import localcontext

import pytest

from transformer_gqa_attention_gb300 import _build, abi

U = 2.0 ** -53
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")
SCALINGS = {"plain": {}, "linear": dict(factor=4.0), "bands": dict(factor=8.0, low=1.0, high=4.0, context=8192.0),
            "ramp": dict(factor=16.0, low=1.0, high=32.0, context=4096.0)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def frequency(rot, j, ln, kind, factor=1.0, low=1.0, high=1.0, context=1.0):
    """(radians per position, bound of what a computation in 64 bits is off by); ln: of theta."""
    x = D(2 * j) / D(rot) * ln
    w = (-x).exp()
    own = (2 + (0 if rot & (rot - 1) == 0 else float(x))) * U
    f, c = D(factor), D(context)
    if kind == "plain":
        return w, own * float(w)
    if kind == "linear":
        return w / f, (own + U) * float(w / f)
    if kind == "bands":
        turns = c * w / (2 * PI)
        if turns > D(high):
            return w, own * float(w)
        if turns < D(low):
            return w / f, (own + U) * float(w / f)
        m = (turns - D(low)) / (D(high) - D(low))
        y = (1 - m) * w / f + m * w
        dm = float(turns) / (high - low) * (own + 4 * U) + 4 * U * float(m)
        return y, dm * float(w - w / f) + (own + 4 * U) * float(y)
    at = [D(rot) * (c / (D(n) * 2 * PI)).ln() / (2 * ln) for n in (high, low)]
    a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    m = min(max(D(j - a) / max(D(b - a), D("0.001")), D(0)), D(1))
    y = m * w / f + (1 - m) * w
    return y, 4 * U * float(w - w / f) + (own + 4 * U) * float(y)


@pytest.mark.parametrize("kind", SCALINGS)
@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (112, 500000.0), (96, 10000.0), (48, 1.0e7), (64, 1.0e6), (16, 1.0e6),
                                       (32, 2.0)])
def test_frequencies_to_the_last_bits(rot, theta, kind):
    r = abi.attn_rope_init("pairs", rot, theta, kind, **SCALINGS[kind])
    worst = 0.0
    with localcontext() as digits:
        digits.prec = 60
        ln = D(theta).ln()
        for j in range(rot // 2):
            w, bound = frequency(rot, j, ln, kind, **SCALINGS[kind])
            off = float(abs(D(r.turns[j]) / D(2 ** 64) * 2 * PI - w))
            assert off <= bound + 2 * U * float(w) + 2 * math.pi * 2.0 ** -64, j
            worst = max(worst, off)
    assert worst <= 2.0 ** -51  # of a radian per position: 4.5e-10 at a million
