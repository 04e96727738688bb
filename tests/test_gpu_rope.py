"""GPU parity of the rotary positions against f64.

Bound of an output a' = amplitude (a c - b s): the cosine and sine are off by
at most 2^-22 (the reduced angle is rounded once, 2^-25 of at most pi/4, and
each polynomial step half an ulp of at most 1), two products and a sum round
to f32: (2^-22 + 3 2^-24) amplitude (|a| + |b|) < 2^-21 amplitude (|a| + |b|), then
one rounding to the type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def say(*a):
    print(*a, flush=True)


def reference(x, pos, freqs, layout, amp, inverse):
    """(rotated x in f64, sum |a| + |b| of each output's pair)."""
    x = x.double()
    R = 2 * freqs.numel()
    t = pos.double()[:, None] * freqs.double() * (-1 if inverse else 1)
    c, s = amp * torch.cos(t)[:, None], amp * torch.sin(t)[:, None]
    ia, ib = (torch.arange(R // 2), torch.arange(R // 2) + R // 2) if layout == "half" else \
        (torch.arange(0, R, 2), torch.arange(1, R, 2))
    y, m = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    m[..., ia] = m[..., ib] = a.abs() + b.abs()
    return y, m


def check(name, got, x, pos, freqs, layout, amp, inverse, dt):
    ref, m = reference(x, pos, freqs, layout, amp, inverse)
    e = torch.finfo(dt).eps / 2
    sub = 2.0 ** -25 if dt == torch.float16 else 0.0
    tol = 2.0 ** -21 * amp * m
    tol = tol + e * (ref.abs() + tol) + sub
    R = 2 * freqs.numel()
    assert torch.equal(got[..., R:], x[..., R:])
    err = (got.double() - ref).abs()
    say(f"  {name}: worst {float((err / tol.clamp_min(1e-300)).max()):.3f} of the bound")
    assert bool((err <= tol).all())


def data(T, heads, D, dt, seed):
    return torch.randn((T, heads, D), generator=torch.Generator().manual_seed(seed)).to(dt)


# heads that do and do not fill 16-byte vectors, all or part of a head, one
# token to more than one block per compute unit, grouped and missing k heads
@pytest.mark.parametrize("T,hq,hk,D,R", [(1, 32, 4, 64, 64), (1, 1, 1, 2, 2), (7, 3, 1, 10, 6), (33, 8, 8, 128, 96),
                                         (2000, 4, 1, 80, 80), (5, 2, 0, 34, 34), (130, 5, 2, 66, 2),
                                         (3, 1, 1, 512, 510), (1100, 33, 1, 256, 128)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_parity(qmv, layout, dtype, T, hq, hk, D, R):
    dt = DT[dtype]
    say("rope", layout, dtype, T, hq, hk, D, R)
    q, k = data(T, hq, D, dt, 1), (data(T, hk, D, dt, 2) if hk else None)
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(3))
    f = qmv.rope_freqs(R, device="cpu")
    for inverse, amp in ((False, 1.0), (True, 1.125)):
        qo, ko = qmv.rope(q.cuda(), None if k is None else k.cuda(), pos.cuda(), f.cuda(), layout=layout,
                          amplitude=amp, inverse=inverse)
        check("q", qo.cpu(), q, pos, f, layout, amp, inverse, dt)
        if k is not None:
            check("k", ko.cpu(), k, pos, f, layout, amp, inverse, dt)
        else:
            assert ko is None


def test_far_and_negative_positions(qmv):
    pos = torch.tensor([0, 1, -1, 999983, -1000003, 16777217, 2 ** 31 - 1, -(2 ** 31) + 1])
    q = data(8, 2, 64, torch.float32, 4)
    for f in (qmv.rope_freqs(64, device="cpu"), torch.linspace(0.1, 3.0, 32)):
        qo, _ = qmv.rope(q.cuda(), None, pos.cuda(), f.cuda())
        check("far", qo.cpu(), q, pos, f, "half", 1.0, False, torch.float32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_in_place(qmv, layout):
    """Heads taken out of one fused product, at odd offsets; head-major tensors;
    in place; what lies between stays as it was."""
    T, hq, hk, D, R, dt = 37, 4, 2, 40, 24, torch.bfloat16
    fused = data(T, hq + 2 * hk, D, dt, 5)
    pos, f = torch.arange(T) * 3, qmv.rope_freqs(R, device="cpu")
    dev = fused.cuda()
    qo, ko = qmv.rope(dev[:, :hq], dev[:, hq:hq + hk], pos.cuda(), f.cuda(), layout=layout)
    check("q", qo.cpu(), fused[:, :hq], pos, f, layout, 1.0, False, dt)
    check("k", ko.cpu(), fused[:, hq:hq + hk], pos, f, layout, 1.0, False, dt)
    q, k = dev[:, :hq], dev[:, hq:hq + hk]
    q2, k2 = qmv.rope(q, k, pos.cuda(), f.cuda(), layout=layout, q_out=q, k_out=k)
    assert torch.equal(q2, qo) and torch.equal(k2, ko) and torch.equal(dev[:, hq + hk:].cpu(), fused[:, hq + hk:])
    # [heads][T][D] seen as [T][heads][D], one element past alignment
    flat = torch.zeros(hq * T * D + 1, dtype=dt, device="cuda")
    hm = flat[1:].view(hq, T, D).transpose(0, 1)
    hm.copy_(fused[:, :hq])
    out = torch.empty(hq * T * D + 1, dtype=dt, device="cuda")[1:].view(hq, T, D).transpose(0, 1)
    q3, _ = qmv.rope(hm, None, pos.cuda(), f.cuda(), layout=layout, q_out=out)
    assert torch.equal(q3, qo)


def test_turning_back_and_gradient(qmv):
    """inverse undoes the rotation (amplitude 1), and is its transpose: the inner
    products <rope(x), y> and <x, inverse(y)> agree to f32 rounding."""
    T, D, R = 50, 96, 64
    x, y = data(T, 3, D, torch.float32, 6).cuda(), data(T, 3, D, torch.float32, 7).cuda()
    pos, f = torch.arange(T).cuda() * 1000, qmv.rope_freqs(R)
    a, _ = qmv.rope(x, None, pos, f, amplitude=1.25)
    b, _ = qmv.rope(y, None, pos, f, amplitude=1.25, inverse=True)
    u, v = (a.double() * y.double()).sum(), (x.double() * b.double()).sum()
    assert abs(u - v) <= 2.0 ** -20 * 1.25 * (x.double().abs() * 2).norm() * y.double().norm()
    c, _ = qmv.rope(x, None, pos, f)
    d, _ = qmv.rope(c, None, pos, f, inverse=True)
    assert float((d - x).abs().max()) <= 2 * 2.0 ** -21 * 4 * float(x.abs().max())


def test_infinities_stay_in_their_pair(qmv):
    x = data(4, 2, 16, torch.float32, 8).cuda()
    pos, f = torch.arange(4).cuda() + 1, qmv.rope_freqs(12)
    base, _ = qmv.rope(x, None, pos, f)
    x[1, 0, 2], x[2, 1, 15] = float("inf"), float("nan")
    out, _ = qmv.rope(x, None, pos, f)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[1, 0, 2] = hit[1, 0, 8] = hit[2, 1, 15] = True
    assert torch.equal(out[~hit], base[~hit]) and not torch.isfinite(out[hit]).any()


def test_graph_and_stream(qmv):
    q, k = data(60, 4, 64, torch.bfloat16, 9).cuda(), data(60, 2, 64, torch.bfloat16, 10).cuda()
    pos, f = torch.arange(60).cuda(), qmv.rope_freqs(64)
    base = qmv.rope(q, k, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = qmv.rope(q, k, pos, f, q_out=torch.empty_like(q), k_out=torch.empty_like(k), stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = qmv.rope(q, k, pos, f)
    for _ in range(3):
        g.replay()
        eager = qmv.rope(q, k, pos, f)
        torch.cuda.synchronize()
        for a, b, c, d in zip(base, other, cap, eager):
            assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
        for c in cap:
            c.zero_()


def test_run_together(qmv):
    """The many-token half of a decoder layer: q and k projections (prefill GEMM),
    rotary positions, gated feed-forward; each step against the same step in f64
    on the step's own inputs."""
    import numpy as np
    import oracle
    import workloads as wl
    from gpu_helpers import dev_x, pack_dev
    fmt, M, K, heads, kv, D, F = "w4a16_g64", 90, 256, 4, 2, 64, 320
    wq, wk = wl.gen_weights(fmt, heads * D, K, (41, 0, 0)), wl.gen_weights(fmt, kv * D, K, (41, 0, 1))
    wg, wu = wl.gen_weights(fmt, F, K, (41, 0, 4)), wl.gen_weights(fmt, F, K, (41, 0, 5))
    Xb = wl.gen_x(K, M, "bf16", (41, 0, 0))
    X = dev_x(Xb, "bf16")
    q = qmv.gemm(fmt, pack_dev(qmv, fmt, wq), X, heads * D, K).view(M, heads, D)
    k = qmv.gemm(fmt, pack_dev(qmv, fmt, wk), X, kv * D, K).view(M, kv, D)
    pos, f = torch.arange(M).cuda(), qmv.rope_freqs(D)
    qr, kr = qmv.rope(q, k, pos, f)
    H, G, U = qmv.gemm_glu(fmt, pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu), X, F, K, save=True)
    dX, dG, dU = qmv.gemm_glu_backward(fmt, pack_dev(qmv, fmt, wg), pack_dev(qmv, fmt, wu), G, U, H, F, K)
    check("q", qr.cpu(), q.cpu(), pos.cpu(), f.cpu(), "half", 1.0, False, torch.bfloat16)
    check("k", kr.cpu(), k.cpu(), pos.cpu(), f.cpu(), "half", 1.0, False, torch.bfloat16)
    Xv = oracle.bf16_to_f64(Xb)
    for w, y in ((wq, q.reshape(M, -1)), (wg, G), (wu, U)):
        W = oracle.dequant(fmt, w)
        r = oracle.check_within(y.float().cpu().numpy(), oracle.gemm_ref(W, Xv), oracle.tolerance_bound(W, Xv, 2e-2))
        assert r["ok"], r
    Wg, Wu = (torch.from_numpy(oracle.dequant(fmt, w)).bfloat16().double() for w in (wg, wu))
    ref = dG.cpu().double() @ Wg + dU.cpu().double() @ Wu
    S = dG.cpu().double().abs() @ Wg.abs() + dU.cpu().double().abs() @ Wu.abs()
    tol = 4 * F * 2.0 ** -24 * S
    assert bool(((dX.cpu().double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all())
    assert np.isfinite(dX.float().cpu().numpy()).all()
