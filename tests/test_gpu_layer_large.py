"""The many-token operators on tensors of more than 2^31 values: rows from all of
them against f64, and what lies around those as it was."""
import pytest
import torch

import workloads as wl
from gpu_helpers import pack_dev
from test_gpu_glu import T, act64, check, say, weights

pytestmark = pytest.mark.gpu
e = 2.0 ** -8


def rows_of(M, N):
    """Rows next to the first, the last, and the one where values pass 2^31 (and 2^32 bytes)."""
    r = {0, 1, 63, M // 3, M - 1, M - 2, M - 257}
    for at in (2 ** 31 // N, 2 ** 30 // N):
        r |= {i for i in range(at - 2, at + 3) if 0 <= i < M}
    return torch.tensor(sorted(r))


def randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for i in range(0, shape[0], 1 << 18):
        t[i:i + (1 << 18)].normal_(generator=g)
    return t


# M N past 2^31 with rows that are and are not whole 16-byte pieces, M K past 2^31
@pytest.mark.parametrize("M,N,K", [((1 << 20) + 1001, 2050, 64), ((1 << 20) + 1001, 2056, 64), ((1 << 20) + 1001, 64, 2112)])
def test_gated_products(qmv, M, N, K):
    fmt = "q8_0"
    (wg, Wg), (wu, Wu) = (weights(fmt, N, K, (k, N, K), torch.bfloat16) for k in (95, 96))
    P = pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu)
    X = randn((M, K), 1)
    r = rows_of(M, max(N, K))
    say("forward", M, N, K)
    H, G, U = qmv.gemm_glu(fmt, *P, X, N, K, save=True)
    x = X[r.cuda()].cpu().double()
    g, u = x @ Wg.t(), x @ Wu.t()
    dg, du = (2 * K * T * (x.abs() @ w.abs().t()) for w in (Wg, Wu))
    a = act64("silu", g)[0]
    h = a * u
    pick = [t[r.cuda()].cpu() for t in (H, G, U)]
    check("H", pick[0], h, 1.13 * dg * (u.abs() + du) + a.abs() * du + (2.0 ** -18 + e) * h.abs() * (1 + e))
    check("G", pick[1], g, dg + e * (g.abs() + dg))
    check("U", pick[2], u, du + e * (u.abs() + du))
    for unrounded in (False, True):
        say("backward", M, N, K, unrounded)
        dX, dG, dU = qmv.gemm_glu_backward(fmt, *P, G, U, H, N, K, unrounded=unrounded)
        gr, ur, hr = (t.double() for t in (pick[1], pick[2], pick[0]))
        av, da = act64("silu", gr)
        q = 2.0 ** -18
        fG, fU = hr * ur * da, hr * av
        oG, oU = q * (hr * ur).abs() * (1 + gr.abs()), q * hr.abs() * (1 + gr.abs())
        check("dG", dG[r.cuda()].cpu(), fG, oG + e * (fG.abs() + oG))
        check("dU", dU[r.cuda()].cpu(), fU, oU + e * (fU.abs() + oU))
        dGr, dUr = dG[r.cuda()].cpu().double(), dU[r.cuda()].cpu().double()
        if unrounded:
            oG, oU = oG + e * e * fG.abs(), oU + e * e * fU.abs()
        else:
            fG, fU, oG, oU = dGr, dUr, torch.zeros_like(oG), torch.zeros_like(oU)
        ref = fG @ Wg + fU @ Wu
        off = oG @ Wg.abs() + oU @ Wu.abs() + 8 * N * T * (1 + 2 * e) * (fG.abs() @ Wg.abs() + fU.abs() @ Wu.abs())
        check("dX", dX[r.cuda()].cpu(), ref, off + e * (ref.abs() + off))
        del dX, dG, dU


def test_rope(qmv):
    tokens, heads, D = (1 << 18) + 77, 64, 130
    q = randn((tokens, heads * D), 3).view(tokens, heads, D)
    pos, f = torch.arange(tokens).cuda(), qmv.rope_freqs(128)
    out, _ = qmv.rope(q, None, pos, f)
    r = rows_of(tokens, heads * D)
    a = r.double()[:, None, None] * f.cpu().double()
    x, got = q[r.cuda()].cpu(), out[r.cuda()].cpu()
    u, v = x.double()[..., :64], x.double()[..., 64:128]
    ref = torch.cat((u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()), -1)
    off = 2.0 ** -21 * (u.abs() + v.abs()).repeat(1, 1, 2)
    check("rope", got[..., :128], ref, off + e * (ref.abs() + off))
    assert torch.equal(got[..., 128:], x[..., 128:])
