"""Angles of more turns than f64 counts one by one: the pair is still turned, not
stretched, whatever is left of the angle's own accuracy (2^52 turns and beyond need
frequencies that no model has)."""
import math

import pytest
import torch

from test_gpu_rope_far import exact_angle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lengths_stay(qmv, dtype):
    freqs = torch.tensor([1.0, 3e7, 1e9, 1e20, 1e30, 3.4e38])
    pos = torch.tensor([1, 12345, -999999937, 2 ** 31 - 1])
    x = torch.zeros(4, 1, 12, dtype=dtype)
    x[..., :6] = 1
    y = qmv.rope(x.cuda(), None, pos.cuda(), freqs.cuda())[0].cpu().double()[:, 0]
    c, s = y[:, :6], y[:, 6:]
    e = torch.finfo(dtype).eps / 2
    print(c, s, flush=True)
    assert bool(((c * c + s * s - 1).abs() <= 4 * e + 2.0 ** -20).all())  # both off by e of themselves and 2^-22


def test_below_2_to_the_50(qmv):
    """Up to 2^50 turns (frequencies of 3e6 at far positions) the angle is exact to 2^-45."""
    freqs = torch.tensor([1e4, 1e5, 3e6 - 0.25])
    pos = torch.tensor([2 ** 31 - 1, 2 ** 30 + 12345, -(2 ** 31) + 77])
    x = torch.zeros(3, 1, 6)
    x[..., :3] = 1
    y = qmv.rope(x.cuda(), None, pos.cuda(), freqs.cuda())[0].cpu().double()[:, 0]
    for i, p in enumerate(pos):
        for j, f in enumerate(freqs):
            t = exact_angle(int(p), float(f))
            assert abs(y[i, j].item() - math.cos(t)) <= 2.0 ** -24 and abs(y[i, 3 + j].item() - math.sin(t)) <= 2.0 ** -24
