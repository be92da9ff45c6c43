"""Rotation tables (kvc_rope_tables) up to the last position that there is, against the exact angles of the float64
speeds.

Python's power and quotient are the library's (the C library's, correctly rounded), so that the speeds are the same
numbers; a value is off by the reduced angle's rounding to float32 (at most pi / 4: pi / 4 * 2^-24), the sine's and
cosine's own (1 ulp, 2^-23 at most), the magnitude's rounding and its product's (2^-24 each); by the rate, within 2^-64
of a turn, times a position of 2^31, and by the angle's rounding to 2^-32 of a turn (2^-33 of a turn each)."""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu

PI = Fraction(int("314159265358979323846264338327950288419716939937510582097494459230781640628620899"), 10 ** 80)
LAST = 2 ** 31


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


@pytest.mark.parametrize("dim", [2, 16, 128])
@pytest.mark.parametrize("factor", [1.0, 3.0, 0.125, 1 / 1024, 2.0 ** -20])
@pytest.mark.parametrize("first,n", [(LAST - 65, 65), (LAST - 1, 1), (3 * 2 ** 27 + 5, 40)])
def test_far_positions(K, dim, factor, first, n):
    base = 10000.0
    cos, sin = torch.full((2, n, dim // 2), 7.0, device="cuda")
    K.kvc_rope_tables(cos, sin, first=first, base=base, scaling=K.KVC_ROPE_LINEAR, factor=factor)
    cos, sin = cos.tolist(), sin.tolist()
    bound = (math.pi / 4 + 4) * 2.0 ** -24 + 2 * math.pi * 2.0 ** -32
    for i in range(dim // 2):
        speed = Fraction(base ** (-2.0 * i / dim) / factor)
        for p in {0, n // 2, n - 1}:
            turns = (first + p) * speed / (2 * PI)
            angle = float((turns - int(turns)) * 2 * PI)
            assert abs(cos[p][i] - math.cos(angle)) <= bound, (i, p)
            assert abs(sin[p][i] - math.sin(angle)) <= bound, (i, p)


def test_one_position_more(K):
    cos, sin = torch.zeros((2, 2, 8), device="cuda")
    with pytest.raises(K.KvcError, match="SHAPE"):
        K.kvc_rope_tables(cos, sin, first=LAST - 1)
