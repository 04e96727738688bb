"""What a rotary pair of an f32 head is multiplied by, amplitude cos t and amplitude
sin t, is rounded to f32 once.

With a = 1, b = 0 a pair comes out as these two: half a step of the value, 2^-24 of
it, and 2^-33 for the f64 arithmetic (its polynomials end below 2^-39).  The f32 heads
of a whole call are then off by at most this of amplitude (|a| + |b|), two products
and a sum.
"""
import math

import pytest
import torch

from test_gpu_rope_far import exact_angle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("amplitude", [1.0, 1.125, float(torch.tensor(1.1386294)), 0.7])
def test_rounded_once(qmv, amplitude, inverse):
    R, T = 64, 128
    amp = float(torch.tensor(amplitude, dtype=torch.float32))  # the call takes it as f32
    pos, f = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(1)), qmv.rope_freqs(R, device="cpu")
    x = torch.zeros(T, 1, R)
    x[..., :R // 2] = 1
    y = qmv.rope(x.cuda(), None, pos.cuda(), f.cuda(), amplitude=amp, inverse=inverse)[0].cpu().double()[:, 0]
    t = [[exact_angle(int(p), float(v)) for v in f] for p in pos]
    c = torch.tensor([[amp * math.cos(v) for v in r] for r in t], dtype=torch.float64)
    s = torch.tensor([[(-amp if inverse else amp) * math.sin(v) for v in r] for r in t], dtype=torch.float64)
    for name, got, want in (("cos", y[:, :R // 2], c), ("sin", y[:, R // 2:], s)):
        off = (got - want).abs() / (2.0 ** -24 * want.abs() + 2.0 ** -33)
        print(f"  {name}: worst {float(off.max()):.3f} of half a step", flush=True)
        assert bool((off <= 1).all())


def test_f32_heads(qmv):
    """The error of an f32 call against one that rounds only its result: with exact
    factors rounded once, each of two products, the sum and both factors give half
    a step at most, 3 2^-24 amplitude (|a| + |b|) together."""
    R, T, amp = 128, 300, 1.1386294
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, 3, R, generator=g)
    pos, f = torch.randint(0, 8192, (T,), generator=g), qmv.rope_freqs(R, device="cpu")
    y = qmv.rope(x.cuda(), None, pos.cuda(), f.cuda(), amplitude=amp)[0].cpu().double()
    a32 = float(torch.tensor(amp, dtype=torch.float32))
    t = torch.tensor([[exact_angle(int(p), float(v)) for v in f] for p in pos], dtype=torch.float64)[:, None]
    a, b = x.double()[..., :R // 2], x.double()[..., R // 2:]
    c, s = a32 * t.cos(), a32 * t.sin()
    ref = torch.cat((a * c - b * s, b * c + a * s), -1)
    m = (a.abs() + b.abs()).repeat(1, 1, 2)
    worst = float(((y - ref).abs() / (3.01 * 2.0 ** -24 * a32 * m)).max())
    print(f"  worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1
