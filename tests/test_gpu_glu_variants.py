"""Every variant of the gated products' forward kernels in every format and type,
with several turns of its loops: the waits of a tile's copies are a constant of
its own for each format and tile.  References and bounds as in test_gpu_glu.py (f64
products on the GPU)."""
import functools

import pytest
import torch

import workloads as wl
from glu_variants import CASES, forward_variant, k_of
from gpu_helpers import pack_dev
from test_gpu_glu import DT, T, act64, check, half_step, inputs, say, weights

pytestmark = pytest.mark.gpu


@functools.lru_cache(maxsize=4)
def matrices(qmv, fmt, N, K, dtype):
    out = []
    for key in (81, 82):
        w, W = weights(fmt, N, K, (key, N, K), DT[dtype])
        out.append((pack_dev(qmv, fmt, w), W.cuda()))
    return out


@pytest.mark.parametrize("M,N,least", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_forward(qmv, fmt, dtype, M, N, least):
    K, dt = k_of(least, wl.BLOCK[fmt]), DT[dtype]
    act = ("silu", "gelu_tanh", "gelu")[(M + wl.FORMATS.index(fmt)) % 3]
    say("glu", fmt, dtype, act, M, N, K, forward_variant(M, N, K))
    (Pg, Wg), (Pu, Wu) = matrices(qmv, fmt, N, K, dtype)
    X = inputs((M, K), dt, M).cuda()
    H, G, U = qmv.gemm_glu(fmt, Pg, Pu, X, N, K, act=act, save=True)
    e, sub = half_step(dt)
    x = X.double()
    g, u = x @ Wg.t(), x @ Wu.t()
    dg, du = 2 * K * T * (x.abs() @ Wg.abs().t()), 2 * K * T * (x.abs() @ Wu.abs().t())
    a = act64(act, g)[0]
    h = a * u
    check("H", H, h, 1.13 * dg * (u.abs() + du) + a.abs() * du + (2.0 ** -18 + e) * h.abs() * (1 + e) + sub)
    check("G", G, g, dg + e * (g.abs() + dg) + sub)
    check("U", U, u, du + e * (u.abs() + du) + sub)
    again = qmv.gemm_glu(fmt, Pg, Pu, X, N, K, act=act)  # without G and U, and bit for bit
    assert torch.equal(again, H)
