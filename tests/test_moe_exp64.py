"""The router's exponential in fp64 (no GPU): its steps as the source has them, with its
constants, every fma rounded once, against 60 digits."""
from __future__ import annotations

import math
import random
import re
from decimal import Decimal, getcontext
from fractions import Fraction
from pathlib import Path

import pytest

SOURCE = Path(__file__).resolve().parents[1] / "dense_block_scaled_amd" / "csrc" / "moe_route.hip"


def _constants():
    text = SOURCE.read_text()
    body = text[text.index("double exp64(double x)"):]
    body = body[:body.index("\n}\n")]
    number = r"[-+0-9.e]+"
    (round_,), (log2e,), (p,) = (re.findall(rf"{name} = ({number});", body) for name in ("kRound", "kLog2e", "double p"))
    c = [float(v) for v in re.search(r"c\[9\] = \{([^}]*)\}", body).group(1).split(",")]
    assert len(c) == 9 and "__builtin_fma(x, kLog2e, kRound)" in body and "__builtin_fma(x, kLog2e, -(shifted - kRound))" in body
    return float(round_), float(log2e), [float(p), *c]


def _fma(a: float, b: float, c: float) -> float:
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def _off(x: float, constants) -> float:
    round_, log2e, c = constants
    n = _fma(x, log2e, round_) - round_
    f = _fma(x, log2e, -n)
    assert n == int(n) and abs(f) <= 0.5 + 2.0 ** -40
    p = c[0]
    for v in c[1:]:
        p = _fma(p, f, v)
    got = Fraction(p) * Fraction(2) ** int(n)
    getcontext().prec = 60
    return abs(float(Decimal(got.numerator) / Decimal(got.denominator) / Decimal(x).exp() - 1))


@pytest.mark.parametrize("lo,hi,bound", [(0, 1, -45.5), (1, 60, -45.5), (60, 300, -45.3), (300, 708, -44.9)])
def test_exponential_is_as_near_as_it_says(lo, hi, bound):
    constants = _constants()
    rng = random.Random(lo)
    xs = [s * rng.uniform(lo, hi) for s in (1, -1) for _ in range(1500)] + [lo, -lo, hi, -hi]
    # the ends of |f| <= 1 / 2, where the polynomial is furthest off
    xs += [s * (n + 0.5) * math.log(2) for s in (1, -1) for n in range(math.ceil(lo / math.log(2)), int(hi / math.log(2)))]
    assert max(_off(float(x), constants) for x in xs) < 2.0 ** bound
