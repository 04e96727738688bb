"""Weights that are infinite in the operand type (f16: past 65504): dX has the
infinities and the NaNs that its formula gives, and no others.  The rows with
such weights are the matrices' last, next to the rows and the stages that only
fill up a tile.

Reference: f64 sums over the returned dG and dU, in which infinite weights give
infinities by themselves; the finite rest within the bound of test_gpu_glu.py.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from gpu_helpers import pack_dev
from test_gpu_glu import DT, T, check, half_step, inputs, say, weights

pytestmark = pytest.mark.gpu


def with_infinite_row(fmt, N, K, key, dt, row):
    """Packed-able arrays whose weights of one row are past the type's range
    (dense: a few of them infinite), and W~ in f64."""
    w, _ = weights(fmt, N, K, key, dt)
    if fmt == "bf16":
        w["q"][row, [0, 5, K - 1]] = 0x7F80  # +inf
        w["q"][row, 9] = 0xFF80
    else:
        f = "d" if "d" in w else "scale"
        if w[f].dtype == np.uint16:
            w[f][row] = np.float16(60000).view(np.uint16)
        else:
            w[f][row] = 1e6
        if "dmin" in w:
            w["dmin"][row] = 0
    W = torch.from_numpy(oracle.dequant(fmt, w)).to(dt).double()
    assert bool(torch.isinf(W[row]).any()) and bool(torch.isfinite(W[[i for i in range(N) if i != row]]).all())
    return w, W


def run(qmv, fmt, dtype, M, N, K, up, row):
    dt = DT[dtype]
    say("glu_bwd infinite", fmt, dtype, M, N, K, "up" if up else "gate", row)
    bad = with_infinite_row(fmt, N, K, (61, N, K), dt, row)
    good = weights(fmt, N, K, (62, N, K), dt)
    (wg, Wg), (wu, Wu) = (good, bad) if up else (bad, good)
    P = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    G, U, dH = (inputs((M, N), dt, 31 + i).cuda() for i in range(3))
    dX, dG, dU = (t.cpu() for t in qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K))
    ref = dG.double() @ Wg + dU.double() @ Wu
    assert bool(torch.isinf(ref).any())
    say("  infinite", int(torch.isinf(ref).sum()), "nan", int(torch.isnan(ref).sum()), "got", int(torch.isinf(dX).sum()),
        int(torch.isnan(dX).sum()))
    # a finite sum may round to an infinity too; next to that border (the bound below
    # is far less than 1 / 64) either is right
    clear = ~((ref.abs() / torch.finfo(dt).max - 1).abs() < 1 / 64)
    want = ref.to(dt)
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(dX)[clear], f(want)[clear])
    ok = torch.isfinite(want) & clear
    zero = torch.zeros(())
    S = dG.double().abs() @ Wg.abs() + dU.double().abs() @ Wu.abs()
    e, sub = half_step(dt)
    d = 4 * N * T * torch.where(ok, S, zero)
    r = torch.where(ok, ref, zero)
    check("dX", torch.where(ok, dX, zero.to(dt)), r, d + e * (r.abs() + d) + sub)
    wide = qmv.gemm_glu_backward(fmt, *P, G, U, dH, N, K, unrounded=True)[0].cpu()
    # with low parts: infinite or NaN there, finite elsewhere
    assert torch.equal(torch.isfinite(wide)[clear], ok[clear])


# N inside a stage; six and ten stages: a padded turn of four behind the last
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("N", [70, 130])
@pytest.mark.parametrize("fmt,dtype", [(f, "f16") for f in wl.FORMATS] + [("bf16", "bf16")])
def test_last_row(qmv, fmt, dtype, N, up):
    run(qmv, fmt, dtype, 40, N, max(128, wl.BLOCK[fmt]), up, N - 1)


# a last stage that is whole, and a row in its middle
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("fmt,dtype", [("w4a16_g64", "f16"), ("q6k", "f16"), ("bf16", "f16"), ("bf16", "bf16")])
def test_padded_stages(qmv, fmt, dtype, up):
    run(qmv, fmt, dtype, 33, 96, 256, up, 96 - 20)


# the middle and the large tile
@pytest.mark.parametrize("fmt,dtype", [("w4a16_g64", "f16"), ("bf16", "f16"), ("bf16", "bf16")])
def test_larger_tiles(qmv, fmt, dtype):
    run(qmv, fmt, dtype, 9000, 190, 512, True, 189)
    run(qmv, fmt, dtype, 2050, 500, 4160, False, 499)


@pytest.mark.parametrize("M", [1, 40, 200])
@pytest.mark.parametrize("fmt,dtype", [("q8_0", "f16"), ("bf16", "bf16")])
def test_forward(qmv, fmt, dtype, M):
    """An infinite gate row reaches its own column of G and H only."""
    dt, N, K = DT[dtype], 70, 96
    wg, Wg = with_infinite_row(fmt, N, K, (63, N, K), dt, N - 1)
    wu, Wu = weights(fmt, N, K, (64, N, K), dt)
    X = inputs((M, K), dt, 35)
    H, G, U = (t.cpu() for t in qmv.gemm_glu(fmt, pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu), X.cuda(), N, K, save=True))
    assert not bool(torch.isfinite(G[:, N - 1]).any())
    assert bool(torch.isfinite(G[:, :N - 1]).all() & torch.isfinite(H[:, :N - 1]).all() & torch.isfinite(U).all())
