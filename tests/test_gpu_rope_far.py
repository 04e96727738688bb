"""Cosines and sines of far positions, against exact arithmetic.

pos * freq is a product of whole numbers and powers of two; here it is reduced by a
2 pi of 200 bits in whole numbers, so the reference angle is not rounded before
its sine is taken (a product of two f64 would round it: 31 + 24 bits).  With
a = 1, b = 0 a pair comes out as (cos, sin).  They are off by at most 2^-22: the
reduced angle is rounded once, 2^-25, and every step of a polynomial by at most
half an ulp of 1.
"""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
BITS = 260


def arctan_inverse(n):  # 2^BITS atan(1 / n)
    x = (1 << (BITS + 20)) // n
    s, k, sign = x, 1, -1
    while x:
        x //= n * n
        k += 2
        s += sign * (x // k)
        sign = -sign
    return s >> 20


TWO_PI = 2 * 4 * (4 * arctan_inverse(5) - arctan_inverse(239))  # Machin


def exact_angle(pos, freq):
    """pos * freq (freq a float) less the nearest whole turns, rounded to f64 once."""
    num, den = float(freq).as_integer_ratio()
    t = pos * num * (1 << BITS)
    t = t // den if den & (den - 1) else t >> (den.bit_length() - 1)
    turns = (2 * t + TWO_PI) // (2 * TWO_PI)
    return (t - turns * TWO_PI) / (1 << BITS)


def test_reference():
    assert abs(TWO_PI / (1 << BITS) - 2 * math.pi) < 1e-15
    for pos in (0, 1, 5, -7, 1000):
        d = exact_angle(pos, 0.5) - pos * 0.5
        assert abs(d / (2 * math.pi) - round(d / (2 * math.pi))) < 1e-13


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("top", [12, 20, 26, 31])
def test_cos_and_sin(qmv, top, layout):
    rng = random.Random(top)
    R, T = 64, 96
    pos = [rng.choice((-1, 1)) * rng.randrange(1 << (top - 1), 1 << top) for _ in range(T - 2)] + [0, (1 << top) - 1]
    for freqs in (qmv.rope_freqs(R, device="cpu"), torch.rand(R // 2, generator=torch.Generator().manual_seed(top)) * 3):
        x = torch.zeros(T, 1, R)
        if layout == "half":
            x[..., :R // 2] = 1
        else:
            x[..., 0::2] = 1
        y = qmv.rope(x.cuda(), None, torch.tensor(pos).cuda(), freqs.cuda(), layout=layout)[0].cpu().double()[:, 0]
        c, s = (y[:, :R // 2], y[:, R // 2:]) if layout == "half" else (y[:, 0::2], y[:, 1::2])
        t = [[exact_angle(p, float(f)) for f in freqs] for p in pos]
        worst = max(max(abs(c[i, j].item() - math.cos(t[i][j])), abs(s[i, j].item() - math.sin(t[i][j])))
                    for i in range(T) for j in range(R // 2))
        print(f"  |pos| < 2^{top}: worst {worst:.3g}, {worst * 2 ** 22:.3f} of the bound", flush=True)
        assert worst <= 2.0 ** -22
