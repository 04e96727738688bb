"""GPU parity of the gated products' backward pass with dX summed over dG and dU
as they are before their rounding (unrounded=True).

Reference: f64 from the given G, U, dH and the weights rounded once to the 16-bit
type.  With e = eps / 2 of the type and t = 2^-24:
  an operand   its f32 value is off by 2^-18 (1 + |g|) of |dh u| (dG) or of |dh| (dU),
               as in the rounded form, and its two 16-bit parts leave e of e of it (in
               f16 also half of 2^-24, where the low part ends)
  dX           these against |W~|, then 4 N products (two parts, two matrices) added in
               f32 in any order, 2 (4 N) t S with S = sum (1 + e) |dG| |W~g| + (1 + e) |dU| |W~u|,
               and one rounding
  dG, dU       the same bits as without unrounded
The sum over the rounded dG and dU misses this bound wherever a sum is small
against its terms, which the first test shows.
"""
import pytest
import torch

import workloads as wl
from gpu_helpers import pack_dev
from test_gpu_glu import DT, T, act64, check, half_step, inputs, say, weights

pytestmark = pytest.mark.gpu


def case(qmv, fmt, dtype, act, M, N, K, scale=0.25):
    dt = DT[dtype]
    say("glu_bwd unrounded", fmt, dtype, act, M, N, K)
    (wg, Wg), (wu, Wu) = weights(fmt, N, K, (53, N, K), dt), weights(fmt, N, K, (54, N, K), dt)
    G, U, dH = inputs((M, N), dt, 21), inputs((M, N), dt, 22), inputs((M, N), dt, 23, scale)
    g, u, dh = G.double(), U.double(), dH.double()
    a, da = act64(act, g)
    dG, dU = dh * u * da, dh * a
    e, sub = half_step(dt)
    r = 2.0 ** -18 * (1 + g.abs())
    off_g = r * (dh * u).abs() + e * e * dG.abs() + sub
    off_u = r * dh.abs() + e * e * dU.abs() + sub
    ref = dG @ Wg + dU @ Wu
    S = (1 + e) * (dG.abs() @ Wg.abs() + dU.abs() @ Wu.abs())
    off = off_g @ Wg.abs() + off_u @ Wu.abs()
    off = off + 8 * N * T * (S + off)
    tol = off + e * (ref.abs() + off) + sub
    P = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    return P, (G.cuda(), U.cuda(), dH.cuda()), ref, tol


def run(qmv, fmt, dtype, act, M, N, K, scale=0.25, alias=False):
    P, (G, U, dH), ref, tol = case(qmv, fmt, dtype, act, M, N, K, scale)
    _, dG0, dU0 = qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K, act=act)
    # a workspace of NaNs shows what is read without having been written
    ws = torch.full((qmv.gemm_glu_backward_bytes(fmt, N, K, M, unrounded=True) + 64,), 255, dtype=torch.uint8, device="cuda")
    kw = dict(dG=dH, dU=G) if alias else {}
    dX, dG, dU = qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K, act=act, workspace=ws[:-64], unrounded=True, **kw)
    torch.cuda.synchronize()
    assert torch.equal(dG, dG0) and torch.equal(dU, dU0)
    assert bool((ws[-64:] == 255).all())
    check("dX", dX.cpu(), ref, tol)
    return dX.cpu(), ref


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_error_of_one_rounding(qmv, dtype):
    """dX is off by no more than its own rounding and a hundredth (the parts leave
    2^-16 of an operand or less), and the sum over the rounded dG and dU by more,
    on most elements' scale and past the bound of this file."""
    fmt, M, N, K, dt = "w4a16_g64", 96, 160, 256, DT[dtype]
    P, (G, U, dH), ref, tol = case(qmv, fmt, dtype, "silu", M, N, K)
    own = (ref.to(dt).double() - ref).norm()
    wide = qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K, unrounded=True)[0].cpu().double()
    rounded = qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K)[0].cpu().double()
    say("error over one rounding's:", float((wide - ref).norm() / own), float((rounded - ref).norm() / own))
    assert (wide - ref).norm() <= 1.01 * own
    assert bool(((wide - ref).abs() <= tol).all())
    assert (rounded - ref).norm() >= 1.3 * own and bool(((rounded - ref).abs() > tol).any())


# as in the rounded form: one to many tokens, N not a multiple of 8 or of a stage,
# K below, at and past the tile, with and without split sums
@pytest.mark.parametrize("M,N,mult", [(1, 1, 1), (3, 7, 2), (32, 64, 1), (33, 129, 5), (24, 1000, 2), (130, 70, 3),
                                      (257, 520, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_parity(qmv, fmt, dtype, M, N, mult):
    act = ("silu", "gelu_tanh", "gelu")[(M + mult) % 3]
    run(qmv, fmt, dtype, act, M, N, wl.BLOCK[fmt] * mult, alias=M % 2 == 0)


# the 256 x 256 tile, ragged in every direction, with one cut of the depth and with several
@pytest.mark.parametrize("M,N,K", [(2050, 500, 4160), (2050, 1333, 2112)])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_large_tiles(qmv, fmt, M, N, K):
    if wl.BLOCK[fmt] == 256:
        K = -(-K // 256) * 256
    run(qmv, fmt, "bf16" if wl.FORMATS.index(fmt) % 2 else "f16", "silu", M, N, K)


# the 128 x 128 tile, three turns of the ring; with the depth cut once
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_middle_tiles(qmv, fmt, dtype):
    run(qmv, fmt, dtype, "gelu_tanh", 9000, 190, 512)


def test_middle_tiles_cut(qmv):
    run(qmv, "q4k", "f16", "gelu_tanh", 391, 2731, 1024)


def test_small_gradients(qmv):
    """f16 gradients whose low parts end at 2^-24: within the bound that says so."""
    run(qmv, "w4a16_g64", "f16", "silu", 70, 128, 128, scale=2.0 ** -12)
    run(qmv, "q8_0", "f16", "gelu", 300, 200, 256, scale=2.0 ** -17)


def test_past_the_largest_value(qmv):
    """A dG past the f16 range is an infinity, and so is dX of its row; other rows
    are as they were, a NaN stays in its row too."""
    fmt, M, N, K = "w4a16_g64", 40, 64, 128
    P, (G, U, dH), _, _ = case(qmv, fmt, "f16", "silu", M, N, K)
    base = qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K, unrounded=True)
    U, dH = U.clone(), dH.clone()
    G[3, 7], U[3, 7], dH[3, 7] = 4.0, 1000.0, 1000.0
    dH[9, N - 1] = float("nan")
    out = qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K, unrounded=True)
    keep = [i for i in range(M) if i not in (3, 9)]
    for a, b in zip(out, base):
        assert torch.equal(a[keep], b[keep])
    assert bool(torch.isinf(out[1][3, 7])) and bool(torch.isnan(out[0][9]).all())
    W = qmv.dequant(fmt, P[0], N, K).half()[7]
    assert bool(torch.isinf(out[0][3][W != 0]).all())  # no NaN from the part that is left over


def test_repeats_and_graphs(qmv):
    """Bit for bit the same again, on another stream, and replayed between eager
    calls, in two graphs with workspaces of their own."""
    fmt, M, N, K = "q5k", 100, 300, 512
    P, (G, U, dH), _, _ = case(qmv, fmt, "bf16", "gelu", M, N, K)
    nb = qmv.gemm_glu_backward_bytes(fmt, N, K, M, unrounded=True)

    def call(ws=None, stream=None):
        return qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K, act="gelu", workspace=ws, stream=stream, unrounded=True)

    base = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = call(stream=s)
    s.synchronize()
    graphs = []
    for _ in range(2):
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(ws)
        graphs.append((g, out, ws))
    for _ in range(3):
        for g, out, _ in graphs:
            g.replay()
            eager = call()
            torch.cuda.synchronize()
            for a, b, c, d in zip(out, base, eager, other):
                assert torch.equal(a, b) and torch.equal(c, b) and torch.equal(d, b)
                a.zero_()
