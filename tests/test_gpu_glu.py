"""GPU parity of the gated products of many tokens and of their backward pass.

Reference: f64 products of the exact dequantized weights rounded once to the
16-bit type (the operands of the matrix cores), on the CPU.  With S = sum |x||w|
of an output, e = eps / 2 of the type (one rounding) and t = 2^-24:
  g, u     |err| <= 2 n t S + e |g| (n additions in f32, any order)
  h        1.13 (bound of |act'|) err(g) (|u| + err(u)) + |act(g)| err(u), + 2^-18 |h| for the hardware's exp
           and reciprocal (exp's argument is off by 2^-24 relative, up to |g| of about 40), + e |h|
  dG, dU   elementwise in f32 from given G, U, dH: 2^-18 (1 + |g|) of |dh u| and of |dh| (1 + |g|), + e
  dX       from the returned (rounded) dG, dU: 2 n t S + e |dX|, n = 2 N
f16 results also round to multiples of 2^-24 below 2^-14 (half a step: 2^-25).
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from gpu_helpers import pack_dev

pytestmark = pytest.mark.gpu
T = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def say(*a):
    print(*a, flush=True)


def half_step(dt):
    return torch.finfo(dt).eps / 2, (2.0 ** -25 if dt == torch.float16 else 0.0)


def act64(name, g):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if name == "gelu_tanh":
        c = (2 / torch.pi) ** 0.5
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    p = 0.5 * torch.special.erfc(-g / 2 ** 0.5)
    return g * p, p + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5


def weights(fmt, N, K, key, dt):
    """Packed-able logical arrays of weights of about 1 / sqrt(K), and W~ in f64."""
    w = wl.gen_weights(fmt, N, K, key)
    W32 = oracle.dequant(fmt, w)
    mul = 2.0 ** round(np.log2(1.0 / (np.std(W32) * np.sqrt(K))))  # a power of two keeps the codes' values exact
    for f in ("scale", "d", "dmin"):
        if f in w:
            w[f] = (w[f].view(np.float16).astype(np.float32) * mul).astype(np.float16).view(np.uint16) \
                if w[f].dtype == np.uint16 else (w[f] * np.float32(mul)).astype(np.float32)
    W = torch.from_numpy(oracle.dequant(fmt, w)).to(dt).double()
    return w, W


def inputs(shape, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dt)


def sums(X, W, chunk=512):
    """X W^T and |X| |W|^T in f64."""
    return X @ W.t(), X.abs() @ W.abs().t()


def check(name, got, ref, tol):
    bad = (got.double() - ref).abs() - tol
    worst = float(((got.double() - ref).abs() / tol.clamp_min(1e-300)).max())
    say(f"  {name}: worst {worst:.3f} of the bound")
    assert bool((bad <= 0).all()), (name, worst, int((bad > 0).sum()))


def run_forward(qmv, fmt, dtype, act, M, N, K, save=True):
    dt = DT[dtype]
    say("glu", fmt, dtype, act, M, N, K)
    (wg, Wg), (wu, Wu) = weights(fmt, N, K, (31, N, K), dt), weights(fmt, N, K, (32, N, K), dt)
    X = inputs((M, K), dt, M)
    out = qmv.gemm_glu(fmt, pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu), X.cuda(), N, K, act=act, save=save)
    torch.cuda.synchronize()
    H, G, U = (t.cpu() for t in out) if save else (out.cpu(), None, None)
    e, sub = half_step(dt)
    g, Sg = sums(X.double(), Wg)
    u, Su = sums(X.double(), Wu)
    a, _ = act64(act, g)
    dg, du = 2 * K * T * Sg, 2 * K * T * Su
    h = a * u
    check("H", H, h, 1.13 * dg * (u.abs() + du) + a.abs() * du + (2.0 ** -18 + e) * h.abs() * (1 + e) + sub)
    if save:
        check("G", G, g, dg + e * (g.abs() + dg) + sub)
        check("U", U, u, du + e * (u.abs() + du) + sub)


# every kernel variant: up to 16, 32, 64 tokens (one weight stream), ragged
# tiles past that, K of one unit, half a step and more than one
@pytest.mark.parametrize("M,N,mult", [(1, 40, 1), (16, 33, 3), (17, 130, 2), (31, 16, 1), (50, 77, 5), (64, 96, 1),
                                      (65, 63, 3), (129, 200, 2), (300, 65, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_forward(qmv, fmt, dtype, M, N, mult):
    act = ("silu", "gelu_tanh", "gelu")[(M + mult) % 3]
    run_forward(qmv, fmt, dtype, act, M, N, wl.BLOCK[fmt] * mult, save=M % 2 == 1)


@pytest.mark.parametrize("fmt,dtype,act,M,N,K", [
    ("w4a16_g64", "bf16", "silu", 1, 5632, 2048), ("q4k", "f16", "gelu", 16, 5632, 2048),
    ("q6k", "bf16", "silu", 512, 1408, 2048), ("bf16", "bf16", "silu", 1030, 700, 1056),
    # one round of 64 x 128 and of 64 x 256 tiles, and two to a unit, ragged in every direction
    ("w4a16_g64", "bf16", "silu", 250, 5000, 320), ("q5_0", "f16", "gelu", 250, 5000, 352),
    ("bf16", "f16", "silu", 500, 5000, 288), ("q6k", "bf16", "gelu_tanh", 500, 5000, 256),
    ("q8_0", "bf16", "silu", 600, 5600, 544), ("q4k", "f16", "silu", 600, 5600, 512),
    # enough 256-token tiles for the large kernel, ragged in every direction
    ("w4a16_g64", "bf16", "silu", 4100, 2050, 192), ("q8_0", "f16", "gelu_tanh", 4100, 2050, 96),
    ("q5k", "bf16", "gelu", 4100, 2050, 256), ("bf16", "f16", "silu", 4100, 2050, 64)])
def test_forward_sizes(qmv, fmt, dtype, act, M, N, K):
    run_forward(qmv, fmt, dtype, act, M, N, K)


# the 64 x 64 tile, ragged in both directions: from K = 1024 on two groups of
# waves share its depth (here of unequal halves, with and without units past the
# last whole run), below one does all of it
@pytest.mark.parametrize("least", [1280, 1024, 512, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_forward_small_tiles(qmv, fmt, dtype, least):
    K = least if wl.BLOCK[fmt] == 256 else least + (96 if wl.BLOCK[fmt] == 32 else 64)
    act = ("silu", "gelu_tanh", "gelu")[wl.FORMATS.index(fmt) % 3]
    run_forward(qmv, fmt, dtype, act, 200, 1333, max(K, wl.BLOCK[fmt]), save=least == 1280)


def run_backward(qmv, fmt, dtype, act, M, N, K, alias=False, scale=0.25):
    dt = DT[dtype]
    say("glu_bwd", fmt, dtype, act, M, N, K)
    (wg, Wg), (wu, Wu) = weights(fmt, N, K, (33, N, K), dt), weights(fmt, N, K, (34, N, K), dt)
    G, U, dH = inputs((M, N), dt, 1), inputs((M, N), dt, 2), inputs((M, N), dt, 3, scale)
    Gd, Ud, Hd = G.cuda(), U.cuda(), dH.cuda()
    kw = dict(dG=Gd, dU=Hd) if alias else {}
    dX, dG, dU = qmv.gemm_glu_backward(fmt, pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu), Gd, Ud, Hd, N, K, act=act, **kw)
    torch.cuda.synchronize()
    dX, dG, dU = dX.cpu(), dG.cpu(), dU.cpu()
    e, sub = half_step(dt)
    g, u, dh = G.double(), U.double(), dH.double()
    a, da = act64(act, g)
    r = 2.0 ** -18
    check("dG", dG, dh * u * da, r * (dh * u).abs() * (1 + g.abs()) + e * (dh * u * da).abs() * (1 + r) + sub)
    check("dU", dU, dh * a, r * dh.abs() * (1 + g.abs()) + e * (dh * a).abs() * (1 + r) + sub)
    ref = dG.double() @ Wg + dU.double() @ Wu
    S = dG.double().abs() @ Wg.abs() + dU.double().abs() @ Wu.abs()
    d = 4 * N * T * S
    check("dX", dX, ref, d + e * (ref.abs() + d) + sub)


# one to many tokens, N not a multiple of 8 (rows of any alignment) or of the
# 64-row step, K below, at and past the tile, with and without split sums
@pytest.mark.parametrize("M,N,mult", [(1, 1, 1), (3, 7, 2), (32, 64, 1), (33, 129, 5), (24, 1000, 2), (130, 70, 3),
                                      (257, 520, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_backward(qmv, fmt, dtype, M, N, mult):
    act = ("silu", "gelu_tanh", "gelu")[(M + mult) % 3]
    run_backward(qmv, fmt, dtype, act, M, N, wl.BLOCK[fmt] * mult, alias=M % 2 == 0)


@pytest.mark.parametrize("fmt,dtype,act,M,N,K", [
    ("bf16", "bf16", "silu", 24, 5632, 2048), ("q4k", "f16", "gelu_tanh", 391, 2731, 1024),
    # the large kernel
    ("w4a16_g64", "bf16", "silu", 4100, 200, 4160), ("q6k", "f16", "gelu", 4100, 67, 4352),
    ("i8row", "bf16", "silu", 4100, 136, 4128)])
def test_backward_sizes(qmv, fmt, dtype, act, M, N, K):
    run_backward(qmv, fmt, dtype, act, M, N, K)


# the 256 x 256 tile, ragged in every direction, with one cut of the depth and with several
@pytest.mark.parametrize("M,N,K", [(2050, 500, 4160), (2050, 1333, 2112)])
@pytest.mark.parametrize("fmt", wl.FORMATS)
def test_backward_large_tiles(qmv, fmt, M, N, K):
    if wl.BLOCK[fmt] == 256:
        K = -(-K // 256) * 256
    run_backward(qmv, fmt, "f16" if wl.FORMATS.index(fmt) % 2 else "bf16", "silu", M, N, K)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_gradient_against_differences(qmv, act):
    """The whole pass (forward with saved products, backward) against central
    differences of the f64 forward of the same W~: L = sum(H dH), along two
    directions.  Rounding of G, U, dG, dU and dX to bf16 is up to e each, on
    sums of terms of both signs: 8 e of the norms' product bounds it."""
    fmt, M, N, K, dt = "w4a16_g64", 40, 96, 128, torch.bfloat16
    (wg, Wg), (wu, Wu) = weights(fmt, N, K, (35, 0, 0), dt), weights(fmt, N, K, (36, 0, 0), dt)
    Pg, Pu = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    X, dH = inputs((M, K), dt, 5), inputs((M, N), dt, 6)
    H, G, U = qmv.gemm_glu(fmt, Pg, Pu, X.cuda(), N, K, act=act, save=True)
    dX, _, _ = qmv.gemm_glu_backward(fmt, Pg, Pu, G, U, dH.cuda(), N, K, act=act)
    dX = dX.cpu().double()

    def loss(x):
        return (act64(act, x @ Wg.t())[0] * (x @ Wu.t()) * dH.double()).sum()

    for seed in (7, 8):
        E = torch.randn((M, K), generator=torch.Generator().manual_seed(seed)).double()
        t = 1e-5
        num = (loss(X.double() + t * E) - loss(X.double() - t * E)) / (2 * t)
        got = (dX * E).sum()
        say(act, float(num), float(got))
        assert abs(num - got) <= 8 * 2.0 ** -8 * dX.norm() * E.norm()


def test_large_arguments(qmv):
    """Saturated activations: finite, and their limits."""
    fmt, N, K, M = "bf16", 32, 32, 64
    W = torch.zeros(N, K)
    W[torch.arange(32), torch.arange(32)] = 1.0
    P = pack_dev(qmv, fmt, {"q": wl.to_bf16_bits(W.numpy())})
    X = torch.zeros(M, K)
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 90.0, -90.0, 1e4, -1e4, 1e18, -1e18])
    X[:, :12] = vals
    X = X.bfloat16()
    for act in ("silu", "gelu_tanh", "gelu"):
        H, G, U = qmv.gemm_glu(fmt, P, P, X.cuda(), N, K, act=act, save=True)
        assert torch.equal(G.cpu(), X) and torch.equal(U.cpu(), X)
        g = X.double()
        h = act64(act, g)[0] * g
        ref = torch.where(g.abs() >= 90, torch.where(g > 0, g * g, 0.0), h)  # f32: e^-90 g^2 is below any bf16 step of 0
        check(act, H.cpu(), ref, 2.0 ** -8 * ref.abs() * 1.01 + 1e-9)
        one = torch.ones_like(G)
        _, dG, dU = qmv.gemm_glu_backward(fmt, P, P, G, one, one, N, K, act=act)
        a, da = act64(act, g)
        sat = g.abs() >= 90
        check(act + " dU", dU.cpu(), torch.where(sat, g.clamp_min(0), a), 2.0 ** -8 * g.abs() * 1.01 + 1e-9)
        check(act + " dG", dG.cpu(), torch.where(sat, (g > 0).double(), da), 2.0 ** -8 * torch.ones_like(g) * 1.2)


@pytest.mark.parametrize("M", [16, 200])
def test_infinities_stay_in_their_row(qmv, M):
    """An infinity or a NaN of one token reaches no other row, also where K and
    N end inside a tile; rows past M and behind the outputs are not written."""
    fmt, N, K, dt = "q8_0", 70, 96, torch.bfloat16
    (wg, _), (wu, _) = weights(fmt, N, K, (37, 0, 0), dt), weights(fmt, N, K, (38, 0, 0), dt)
    Pg, Pu = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    X = inputs((M, K), dt, 9).cuda()
    base = qmv.gemm_glu(fmt, Pg, Pu, X, N, K, save=True)
    bad = X.clone()
    bad[3, K - 1], bad[5, 0] = float("inf"), float("nan")
    keep = [i for i in range(M) if i not in (3, 5)]
    guard = torch.full((3, M + 4, N), 7.0, dtype=dt, device="cuda")
    # the buffers' rows M .. M + 3 lie behind the call's
    out = qmv.gemm_glu(fmt, Pg, Pu, bad, N, K, H=guard[0, :M], G=torch.empty(M, N, dtype=dt, device="cuda"),
                       U=torch.empty(M, N, dtype=dt, device="cuda"))
    for a, b in zip(out, base):
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(a[3]).any() and torch.isnan(a[5]).all()
    assert bool((guard[0, M:] == 7.0).all())
    G, U, dH = (inputs((M, N), dt, i).cuda() for i in (1, 2, 3))
    base = qmv.gemm_glu_backward(fmt, Pg, Pu, G, U, dH, N, K)
    dB = dH.clone()
    dB[3, N - 1], dB[5, 0] = float("inf"), float("nan")
    out = qmv.gemm_glu_backward(fmt, Pg, Pu, G, U, dB, N, K)
    for a, b in zip(out, base):
        assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(out[0][3]).any() and torch.isnan(out[0][5]).all()


def test_repeats_streams_and_graphs(qmv):
    """Bit for bit the same: again, on another stream, captured and replayed
    between eager calls, two graphs with workspaces of their own."""
    fmt, M, N, K, dt = "q4k", 100, 300, 512, torch.bfloat16
    (wg, _), (wu, _) = weights(fmt, N, K, (39, 0, 0), dt), weights(fmt, N, K, (40, 0, 0), dt)
    Pg, Pu = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    X, dH = inputs((M, K), dt, 1).cuda(), inputs((M, N), dt, 2).cuda()
    nb = qmv.gemm_glu_backward_bytes(fmt, N, K, M)
    assert nb > 0  # the shape takes split sums

    def both(stream=None, ws=None):
        H, G, U = qmv.gemm_glu(fmt, Pg, Pu, X, N, K, save=True, stream=stream)
        return (H, G, U, *qmv.gemm_glu_backward(fmt, Pg, Pu, G, U, dH, N, K, workspace=ws, stream=stream))

    base = [t.clone() for t in both()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for a, b in zip(both(), base):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(ws=ws)
        graphs.append((g, out, ws))
    for _ in range(3):
        for g, out, _ in graphs:
            g.replay()
            eager = both()
            torch.cuda.synchronize()
            for a, b, c in zip(out, base, eager):
                assert torch.equal(a, b) and torch.equal(c, b)
                a.zero_()


def test_small_gradients_keep_their_subnormals(qmv):
    """f16 gradients far below 2^-14: the matrix cores take subnormal operands as
    they are (dX from the returned dG, dU within its bound)."""
    run_backward(qmv, "w4a16_g64", "f16", "silu", 70, 128, 128, scale=2.0 ** -17)
    run_backward(qmv, "bf16", "f16", "gelu", 300, 200, 256, scale=2.0 ** -19)


def test_rounds_of_the_chip(qmv):
    """Backward tiles and cuts at sizes around one round of the chip, against the
    forward's weights: every row of dX equals the row of a one-row call's up to
    the order of its sum."""
    fmt, N, K, dt = "q8_0", 192, 512, torch.bfloat16
    (wg, Wg), (wu, Wu) = weights(fmt, N, K, (43, 0, 0), dt), weights(fmt, N, K, (44, 0, 0), dt)
    Pg, Pu = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    e, _ = half_step(dt)
    for M in (2, 64, 65, 128, 129, 1000, 9000):
        G, U, dH = (inputs((M, N), dt, i) for i in (11, 12, 13))
        dX, dG, dU = (t.cpu() for t in qmv.gemm_glu_backward(fmt, Pg, Pu, G.cuda(), U.cuda(), dH.cuda(), N, K))
        ref = dG.double() @ Wg + dU.double() @ Wu
        d = 4 * N * T * (dG.double().abs() @ Wg.abs() + dU.double().abs() @ Wu.abs())
        say("M", M)
        check("dX", dX, ref, d + e * (ref.abs() + d))


def test_stream_argument_and_devices(qmv):
    """stream= runs there and allocates there; a CPU tensor among them is refused."""
    fmt, M, N, K, dt = "w4a16_g64", 20, 96, 128, torch.bfloat16
    (wg, _), (wu, _) = weights(fmt, N, K, (45, 0, 0), dt), weights(fmt, N, K, (46, 0, 0), dt)
    Pg, Pu = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    X = inputs((M, K), dt, 1).cuda()
    H, G, U = qmv.gemm_glu(fmt, Pg, Pu, X, N, K, save=True)
    base = qmv.gemm_glu_backward(fmt, Pg, Pu, G, U, H, N, K)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qmv.gemm_glu(fmt, Pg, Pu, X, N, K, save=True, stream=s)
    back = qmv.gemm_glu_backward(fmt, Pg, Pu, *got[1:], got[0], N, K, stream=s)
    s.synchronize()
    for a, b in zip((*got, *back), (H, G, U, *base)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        qmv.gemm_glu(fmt, Pg.cpu(), Pu, X, N, K)
    with pytest.raises(ValueError):
        qmv.gemm_glu_backward(fmt, Pg, Pu, G, U.cpu(), H, N, K)
