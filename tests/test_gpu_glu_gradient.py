"""Forward and backward of the gated products together against the gradient of the
f64 forward, so that a term that is left out or wrong shows.

With e = eps / 2 of the type, t = 2^-24 and S the sum of the magnitudes of a product:
  g, u as saved   off by dg = 2 K t S_g + e (|g| + ...), du alike
  dG              |dH| ((|u| + du) c2 dg + (|act'| + c2 dg) du), c2 = 0.85 the bound of |act''|
                  (1/2 for SiLU; 2 / sqrt(2 pi) for GELU, reached at 0), and 2^-18 (1 + |g|) |dH u|
                  for its f32 arithmetic; rounded: e of it; in two parts: e e
  dU              |dH| 1.13 dg and 2^-18 |dH| (1 + |g|), rounded alike
  dX              these against |W~|, the f32 sums, one rounding
"""
import pytest
import torch

from gpu_helpers import pack_dev
from test_gpu_glu import DT, T, act64, check, half_step, inputs, say, weights

pytestmark = pytest.mark.gpu


def whole(qmv, act, dtype, unrounded, fmt="w4a16_g64", M=40, N=96, K=128):
    """dX of the kernels, the f64 gradient's gate and up parts, the bound, the f64 loss."""
    dt = DT[dtype]
    (wg, Wg), (wu, Wu) = weights(fmt, N, K, (91, 0, 0), dt), weights(fmt, N, K, (92, 0, 0), dt)
    Pg, Pu = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    X, dH = inputs((M, K), dt, 51), inputs((M, N), dt, 52)
    H, G, U = qmv.gemm_glu(fmt, Pg, Pu, X.cuda(), N, K, act=act, save=True)
    dX = qmv.gemm_glu_backward(fmt, Pg, Pu, G, U, dH.cuda(), N, K, act=act, unrounded=unrounded)[0].cpu()
    x, dh = X.double(), dH.double()
    g, u = x @ Wg.t(), x @ Wu.t()
    a, da = act64(act, g)
    e, sub = half_step(dt)
    dg, du = (2 * K * T * (x.abs() @ w.abs().t()) for w in (Wg, Wu))
    dg, du = dg + e * (g.abs() + dg) + sub, du + e * (u.abs() + du) + sub
    c2, r, k = 0.85, 2.0 ** -18, e * e if unrounded else e
    dG, dU = dh * u * da, dh * a
    oG = dh.abs() * ((u.abs() + du) * c2 * dg + (da.abs() + c2 * dg) * du) + r * (dh * u).abs() * (1 + g.abs())
    oU = dh.abs() * 1.13 * dg + r * dh.abs() * (1 + g.abs())
    oG, oU = oG + k * (dG.abs() + oG) + sub, oU + k * (dU.abs() + oU) + sub
    S = (dG.abs() + oG) @ Wg.abs() + (dU.abs() + oU) @ Wu.abs()
    off = oG @ Wg.abs() + oU @ Wu.abs() + 8 * N * T * (1 + e) * S
    gate, up = dG @ Wg, dU @ Wu
    tol = off + e * ((gate + up).abs() + off) + sub

    def loss(y):
        return (act64(act, y @ Wg.t())[0] * (y @ Wu.t()) * dh).sum()

    return dX, gate, up, tol, loss, x


@pytest.mark.parametrize("unrounded", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_every_element(qmv, act, dtype, unrounded):
    dX, gate, up, tol, _, _ = whole(qmv, act, dtype, unrounded)
    check("dX", dX, gate + up, tol)
    # what a missing term, or the other's weights, would give is far outside
    for wrong in (gate, up, torch.zeros_like(gate), gate - up):
        assert ((wrong - (gate + up)).abs() > tol).double().mean() > 0.5


@pytest.mark.parametrize("unrounded", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_against_differences(qmv, act, dtype, unrounded):
    """Central differences of the f64 loss along the gradient's own parts, where the
    inner product is the length of the part and not what chance leaves of it."""
    dX, gate, up, tol, loss, x = whole(qmv, act, dtype, unrounded)
    got = dX.double()
    for name, E in (("gate", gate), ("up", up), ("all", gate + up)):
        s = 1e-5 / E.abs().max()
        num = (loss(x + s * E) - loss(x - s * E)) / (2 * s)
        bound = (tol * E.abs()).sum() + 1e-6 * (gate.norm() + up.norm()) * E.norm()  # 1e-6: the step's third order
        say(act, dtype, name, float(num), float((got * E).sum()), "bound", float(bound))
        assert abs((got * E).sum() - num) <= bound
        for part, missing in (("gate", gate), ("up", up)):
            if name in (part, "all"):
                assert abs(((got - missing) * E).sum() - num) > bound, (name, "without", part)
