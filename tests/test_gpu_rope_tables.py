"""Rotation tables (kvc_rope_tables) against their definition in float64.

A table's value is off by: the reduced angle's rounding to float32 (at most pi / 4, so pi / 4 * 2^-24), the sine's
and cosine's own (1 ulp, 2^-23 at most), the magnitude's rounding and its product's (2^-24 each), all times the
magnitude; and by the speed's rounding in float64 (two steps, here and in the definition) times the position."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def speeds(dim, base, scaling, factor, trained, low, high):
    i = torch.arange(dim // 2, dtype=torch.float64)
    if scaling == 2:
        base = base * factor ** (dim / (dim - 2))
    s = base ** (-2 * i / dim)
    if scaling == 1:
        s = s / factor
    if scaling == 3:
        keep = ((trained * s / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        s = keep * s + (1 - keep) * s / factor
    return s


@pytest.mark.parametrize("dim", [2, 6, 16, 48, 64, 128, 250, 256])
@pytest.mark.parametrize("scaling,factor", [(0, 1.0), (1, 4.0), (1, 0.125), (2, 8.0), (3, 16.0)])
@pytest.mark.parametrize("first,n", [(0, 1), (0, 333), (8191, 70), (1 << 24, 65)])
def test_tables(K, dim, scaling, factor, first, n):
    if dim == 2 and scaling == 2:
        pytest.skip("no such base")
    trained, low, high, mag = 4096, 1.0, 32.0, 1.25 if scaling == 3 else 1.0
    base = 500000.0 if scaling else 10000.0
    cos, sin = torch.full((2, n, dim // 2), 7.0, device="cuda")
    K.kvc_rope_tables(cos, sin, first=first, base=base, scaling=scaling, factor=factor, trained=trained, low=low, high=high, magnitude=mag)
    s = speeds(dim, base, scaling, factor, trained, low, high)
    at = (first + torch.arange(n, dtype=torch.float64))[:, None] * s
    bound = mag * ((math.pi / 4 + 2 + 1 + 1) * 2.0 ** -24 + at * 2.0 ** -51)
    for got, want in ((cos, mag * at.cos()), (sin, mag * at.sin())):
        off = (got.cpu().double() - want).abs()
        assert (off <= bound).all(), float((off / bound).max())


def test_quarter_turns(K):
    """A base of 1 and one pair: the angle is the position itself."""
    cos, sin = torch.zeros((2, 100, 1), device="cuda")
    K.kvc_rope_tables(cos, sin, base=1.0, scaling=K.KVC_ROPE_LINEAR, factor=2 / math.pi)  # a quarter turn a position
    p = torch.arange(100)
    want = torch.tensor([[1, 0], [0, 1], [-1, 0], [0, -1]])[p % 4].double()
    assert (cos[:, 0].cpu().double() - want[:, 0]).abs().max() <= 2.0 ** -22
    assert (sin[:, 0].cpu().double() - want[:, 1]).abs().max() <= 2.0 ** -22


def test_refused_and_empty(K):
    cos, sin = torch.zeros((2, 4, 8), device="cuda")
    with pytest.raises(K.KvcError, match="SHAPE"):
        K.kvc_rope_tables(cos, sin, scaling=K.KVC_ROPE_PARTS, factor=2.0, trained=64, low=4.0, high=1.0)
    with pytest.raises(K.KvcError, match="UNSUPPORTED"):
        K.kvc_rope_tables(cos, sin, scaling=9)
    with pytest.raises(ValueError):
        K.kvc_rope_tables(cos, sin.cpu())
    K.kvc_rope_tables(cos[:0], sin[:0])


def test_as_the_calls_take_them(K):
    """The tables of the synthetic workloads."""
    from persistent_kv_cache_gb300 import synth
    want = synth.rope_cache(300, 128)
    cos, sin = torch.zeros((2, 300, 64), device="cuda")
    K.kvc_rope_tables(cos, sin)
    assert (cos.cpu() - want[0]).abs().max() <= 2.0 ** -22 and (sin.cpu() - want[1]).abs().max() <= 2.0 ** -22
