"""Arithmetic of the experts' activations: a value as two e4m3 floats with a power-of-two
scale, restated with torch's e4m3 on the CPU, against what include/e8.h promises of it."""
import math

import pytest
import torch


def _pair(x, amax):
    """hi + lo / 16 in units of s, and s, as the router and the up products write them."""
    e = math.frexp(amax)[1] - 1 + 127 if amax >= 2.0 ** -126 else 0   # exponent field
    s = 2.0 ** ((e - 7 if e > 11 else 4) - 127)
    v = x.double() / s
    hi = v.float().to(torch.float8_e4m3fn).double()
    lo = (16 * (v - hi)).float().to(torch.float8_e4m3fn).double()
    return (hi + lo / 16) * s


def _bf16_from(low, high):
    """Every positive bf16 value in [low, high]."""
    lo, hi = (torch.tensor(v, dtype=torch.float32).view(torch.int32).item() >> 16 for v in (low, high))
    bits = torch.arange(lo, hi + 1, dtype=torch.int32) << 16
    return bits.view(torch.float32).double()


@pytest.mark.parametrize("e", [-133, -130, -126, -120, -117, -116, -115, -100, -1, 0, 7, 100, 126, 127])
@pytest.mark.parametrize("m", [1.0, 1.5, 1.9921875])
def test_tokens(e, m):
    amax = m * 2.0 ** e
    if e < -126:
        amax = 2.0 ** e
    x = _bf16_from(2.0 ** -133, amax)
    off = (_pair(x, amax) - x).abs()
    assert (off[x >= 2.0 ** -13 * amax] == 0).all()
    assert (off <= 2.0 ** -21 * amax).all()
    if amax < 2.0 ** -116:
        assert (off == 0).all()


def test_tokens_are_not_exact_further_down():
    """2^-13 is where it ends: under a largest of 2^7 an odd last place just below is lost."""
    x = torch.tensor([2.0 ** -6 * (1 - 2.0 ** -8)], dtype=torch.float64)
    assert x.bfloat16().double() == x and _pair(x, 128.0) != x


@pytest.mark.parametrize("amax", [1.0, 1.999, 2.0 ** 40, 2.0 ** -115, 2.0 ** -118, 2.0 ** -125])
def test_h(amax):
    g = torch.Generator().manual_seed(1)
    x = (torch.rand(200000, generator=g, dtype=torch.float64) + 1e-9) * 2.0 ** -(18 * torch.rand(200000, generator=g))
    x = (x * amax).clamp(max=amax).float().double()
    off = (_pair(x, amax) - x).abs()
    big = (x >= 2.0 ** -12 * amax) & (x >= 2.0 ** -128)
    assert (off[big] <= 2.0 ** -9 * x[big]).all()
    assert (off[~big] <= max(2.0 ** -21 * amax, 2.0 ** -137)).all()
