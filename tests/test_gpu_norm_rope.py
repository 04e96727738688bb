"""The norms of the q and k heads with their rotary positions, and the gradient,
against f64.

Bounds, in u = 2^-24 (half an f32 step).  The sum of squares: a lane adds at most 40
values one by one and 6 lane sums follow, 46 u of it at most, half of that on the
root; mean, eps, root and reciprocal add 4 u at most: r is off by 27 u.  n = x r and
the weighted n by 3 u more (w + offset is one sum): 30 u.  The rotation adds 8 u
of amplitude (|a| + |b|) (cosine and sine 2^-22 = 4 u, two products and a sum 3 u,
the amplitude's own rounding): y is off by 40 u amplitude (|a| + |b|) with (a, b) the
weighted pair, then one rounding to the type.

Gradient: g is off by 8 u of m = amplitude (|dy_a| + |dy_b|), h = g w by 10 u |w| m;
mean(h n) by (10 + 30 + 46 + 3) u of mean(|w| m |n|), n times it by 30 + 2 u more;
the difference and r by 30 u: dx is off by 130 u r (|w| m + |n| mean(|w| m |n|)),
then one rounding.  dw: every term is off by 40 u of m |n|, and no value passes more
additions than a block has heads (+ 60 for the lanes, waves and blocks).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


def say(*a):
    print(*a, flush=True)


def data(shape, dt, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dt)


def pairs(R, layout):
    if layout == "half":
        return torch.arange(R // 2), torch.arange(R // 2) + R // 2
    return torch.arange(0, R, 2), torch.arange(1, R, 2)


def rot(x, pos, freqs, layout, amp, sign=1):
    """(rotated x, sum |a| + |b| of each value's pair times amp), f64."""
    t = pos.double()[:, None] * freqs.double() * sign
    c, s = amp * torch.cos(t)[:, None], amp * torch.sin(t)[:, None]
    ia, ib = pairs(2 * freqs.numel(), layout)
    y, m = x.clone(), x.abs()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    m[..., ia] = m[..., ib] = amp * (a.abs() + b.abs())
    return y, m


def forward64(x, w, pos, freqs, layout, amp, eps):
    """y and the magnitude its error goes by."""
    n = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    return rot(n * w, pos, freqs, layout, amp)


def half_step(dt):
    return torch.finfo(dt).eps / 2, 2.0 ** -25 if dt == torch.float16 else 0.0


def near(name, got, ref, tol, dt):
    e, sub = half_step(dt)
    tol = tol + e * (ref.abs() + tol) + sub
    err = (got.double().cpu() - ref).abs()
    say(f"  {name}: worst {float((err / tol.clamp_min(1e-300)).max()):.3f} of the bound")
    assert bool((err <= tol).all()), name


def check_forward(name, got, x, w, offset, pos, freqs, layout, amp, eps):
    w64 = (w.double() + offset) if w is not None else torch.ones(x.shape[-1], dtype=torch.float64)
    ref, m = forward64(x.double(), w64, pos, freqs, layout, amp, eps)
    near(name, got, ref, 40 * U * m, x.dtype)


def check_backward(name, got, got_w, x, dy, w, offset, pos, freqs, layout, amp, eps, rows):
    """rows: heads of all tokens that one block adds up."""
    x64 = x.double()
    w64 = (w.double() + offset) if w is not None else torch.ones(x.shape[-1], dtype=torch.float64)
    r = 1 / (x64.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n = x64 * r
    g, m = rot(dy.double(), pos, freqs, layout, amp, -1)
    h, hm = g * w64, m * w64.abs()
    ref = r * (h - n * (h * n).mean(-1, keepdim=True))
    near("d" + name, got, ref, 130 * U * r * (hm + n.abs() * (hm * n.abs()).mean(-1, keepdim=True)), x.dtype)
    if w is None:
        assert got_w is None
        return
    near(f"d{name}_weight", got_w, (g * n).sum((0, 1)), (100 + rows) * U * (m * n.abs()).sum((0, 1)), w.dtype)


# one token to several turns of a block, heads that fill their lanes' pieces and do not, one value
# past a piece, all, part and next to nothing of a head rotated, the largest heads; grouped and missing k
SIZES = [(1, 32, 4, 64, 64), (1, 1, 1, 2, 2), (7, 3, 1, 10, 6), (33, 8, 8, 128, 96), (515, 4, 1, 80, 48),
         (5, 2, 0, 33, 32), (130, 5, 2, 67, 2), (3, 1, 1, 512, 510), (300, 33, 1, 256, 256), (2, 3, 2, 1024, 1024),
         (4, 2, 1, 1023, 6), (19, 40, 40, 16, 8)]


def block_rows(qmv, T, D, heads, count):
    """Heads of tokens that a block of a tensor takes at most (the workspace holds D sums for each block)."""
    blocks = max(1, qmv.norm_rope_backward_bytes(T, D, *heads) // (4 * D) // (2 * len(heads)))
    return -(-T // blocks) * count


@pytest.mark.parametrize("T,hq,hk,D,R", SIZES)
@pytest.mark.parametrize("dtype,w_dtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_parity(qmv, layout, dtype, w_dtype, T, hq, hk, D, R):
    dt, wt = DT[dtype], DT[w_dtype]
    say("norm_rope", layout, dtype, w_dtype, T, hq, hk, D, R)
    q, k = data((T, hq, D), dt, 1, 3.0), (data((T, hk, D), dt, 2) if hk else None)
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(3))
    f = qmv.rope_freqs(R, device="cpu")
    for offset, amp, eps in ((0.0, 1.0, 1e-6), (1.0, 1.125, 1e-2)):
        qw = data((D,), wt, 4, 0.3) + (1 - offset)
        kw = (data((D,), wt, 5, 0.3) + (1 - offset)) if hk else None
        dq, dk = data((T, hq, D), dt, 6, 0.1), (data((T, hk, D), dt, 7) if hk else None)
        on = [None if t is None else t.cuda() for t in (q, k, qw, kw, dq, dk, pos, f)]
        qo, ko = qmv.norm_rope(on[0], on[1], on[2], on[3], on[6], on[7], eps=eps, layout=layout, amplitude=amp,
                               weight_offset=offset)
        gq, gk, gqw, gkw = qmv.norm_rope_backward(*on, eps=eps, layout=layout, amplitude=amp, weight_offset=offset)
        heads = (hq, hk) if hk else (hq,)
        check_forward("q", qo, q, qw, offset, pos, f, layout, amp, eps)
        check_backward("q", gq, gqw, q, dq, qw, offset, pos, f, layout, amp, eps, block_rows(qmv, T, D, heads, hq))
        if hk:
            check_forward("k", ko, k, kw, offset, pos, f, layout, amp, eps)
            check_backward("k", gk, gkw, k, dk, kw, offset, pos, f, layout, amp, eps, block_rows(qmv, T, D, heads, hk))
        else:
            assert ko is None and gk is None and gkw is None


@pytest.mark.parametrize("T,hq,hk,D,R", [(12001, 5, 3, 24, 16), (7003, 35, 1, 10, 10), (70001, 1, 0, 8, 4)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_many_turns_of_a_block(qmv, layout, T, hq, hk, D, R):
    """More tokens than one turn of the blocks that the chip holds: also in place."""
    test_parity(qmv, layout, "bf16", "bf16", T, hq, hk, D, R)
    q = data((T, hq, D), torch.float16, 8).cuda()
    k = data((T, hk, D), torch.float16, 9).cuda() if hk else None
    pos, f = torch.arange(T).cuda(), qmv.rope_freqs(R)
    want = qmv.norm_rope(q, k, None, None, pos, f, layout=layout)
    qmv.norm_rope(q, k, None, None, pos, f, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and (not hk or torch.equal(k, want[1]))


def setup(qmv, T=37, hq=6, hk=2, D=96, R=64, dt=torch.bfloat16):
    q, k = data((T, hq, D), dt, 11).cuda(), data((T, hk, D), dt, 12).cuda()
    qw, kw = ((1 + data((D,), dt, s, 0.3)).cuda() for s in (13, 14))
    dq, dk = data((T, hq, D), dt, 15).cuda(), data((T, hk, D), dt, 16).cuda()
    return q, k, qw, kw, dq, dk, torch.arange(T).cuda() * 31, qmv.rope_freqs(R)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_equals_rope_of_the_norm(qmv, layout):
    """f32: the rotation is qmv.rope's on the normed heads, to the norm's rounding."""
    q, k, qw, kw, _, _, pos, f = setup(qmv, dt=torch.float32)
    a = qmv.norm_rope(q, k, qw, kw, pos, f, layout=layout)
    n = [x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * w for x, w in ((q, qw), (k, kw))]
    b = qmv.rope(*n, pos, f, layout=layout)
    for x, y, z in zip(a, b, n):
        assert float((x - y).abs().max()) <= 2 * 40 * U * 2 * float(z.abs().max())


def test_weights_left_out(qmv):
    q, k, qw, kw, dq, dk, pos, f = setup(qmv)
    one = torch.ones_like(qw)
    a = qmv.norm_rope(q, k, None, None, pos, f, weight_offset=5.0)  # without a weight the offset does not count
    b = qmv.norm_rope(q, k, one, one, pos, f)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = qmv.norm_rope_backward(q, k, None, None, dq, dk, pos, f)
    d = qmv.norm_rope_backward(q, k, one, one, dq, dk, pos, f)
    assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1]) and c[2] is None and c[3] is None
    e = qmv.norm_rope_backward(q, k, qw, kw, dq, dk, pos, f)
    g = qmv.norm_rope_backward(q, k, qw, kw, dq, dk, pos, f, weight_grads=False)
    assert torch.equal(e[0], g[0]) and torch.equal(e[1], g[1]) and g[2] is None and g[3] is None
    h = qmv.norm_rope_backward(q, k, qw, None, dq, dk, pos, f)  # a norm of q alone has a weight
    assert torch.equal(h[0], e[0]) and torch.equal(h[2], e[2]) and torch.equal(h[1], d[1]) and h[3] is None


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_in_place(qmv, layout):
    """Heads out of one fused product, head-major and misaligned tensors, in place: the same values, and what
    lies between stays."""
    T, hq, hk, D, dt = 37, 6, 2, 96, torch.bfloat16
    q, k, qw, kw, dq, dk, pos, f = setup(qmv)
    kw_args = dict(layout=layout)
    ref = qmv.norm_rope(q, k, qw, kw, pos, f, **kw_args)
    back = qmv.norm_rope_backward(q, k, qw, kw, dq, dk, pos, f, **kw_args)
    fused = torch.zeros((T, hq + 2 * hk, D), dtype=dt, device="cuda")
    fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:] = q, k, 7.0
    fq, fk = fused[:, :hq], fused[:, hq:hq + hk]
    got = qmv.norm_rope(fq, fk, qw, kw, pos, f, **kw_args)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    got = qmv.norm_rope_backward(fq, fk, qw, kw, dq, dk, pos, f, **kw_args)
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    flat = torch.zeros(hq * T * D + 1, dtype=dt, device="cuda")
    hm = flat[1:].view(hq, T, D).transpose(0, 1)
    hm.copy_(q)
    out = torch.empty(hq * T * D + 1, dtype=dt, device="cuda")[1:].view(hq, T, D).transpose(0, 1)
    got, _ = qmv.norm_rope(hm, None, qw, None, pos, f, q_out=out, **kw_args)
    assert torch.equal(got, ref[0])
    # the gradient in place: over the gradient it took, over q, and strided
    g2, k2 = dq.clone(), dk.clone()
    got = qmv.norm_rope_backward(q, k, qw, kw, g2, k2, pos, f, dq=g2, dk=k2, **kw_args)
    assert got[0] is g2 and all(torch.equal(a, b) for a, b in zip(got, back))
    got = qmv.norm_rope_backward(fq, fk, qw, kw, dq, dk, pos, f, dq=fq, dk=fk, **kw_args)
    assert all(torch.equal(a, b) for a, b in zip(got, back)) and bool((fused[:, hq + hk:] == 7.0).all())
    fused[:, :hq], fused[:, hq:hq + hk] = q, k
    qmv.norm_rope(fq, fk, qw, kw, pos, f, q_out=fq, k_out=fk, **kw_args)
    assert torch.equal(fq, ref[0]) and torch.equal(fk, ref[1]) and bool((fused[:, hq + hk:] == 7.0).all())


def test_zero_and_special_heads(qmv):
    """A head of zeros gives zeros and a finite gradient; NaN and infinite heads touch no other head."""
    q, k, qw, kw, dq, dk, pos, f = setup(qmv, dt=torch.float32)
    clean = qmv.norm_rope(q, k, qw, kw, pos, f), qmv.norm_rope_backward(q, k, qw, kw, dq, dk, pos, f, weight_grads=False)
    bad = q.clone()
    bad[3, 1] = 0
    bad[5, 2, 7] = float("nan")
    bad[6, 0, 95] = float("inf")
    got = qmv.norm_rope(bad, k, qw, kw, pos, f)[0]
    back = qmv.norm_rope_backward(bad, k, qw, kw, dq, dk, pos, f, weight_grads=False)[0]
    keep = torch.ones(q.shape[:2], dtype=torch.bool)
    keep[3, 1] = keep[5, 2] = keep[6, 0] = False
    assert torch.equal(got[keep], clean[0][0][keep]) and torch.equal(back[keep], clean[1][0][keep])
    assert bool((got[3, 1] == 0).all()) and bool(torch.isfinite(back[3, 1]).all())
    assert bool(torch.isnan(got[5, 2]).all()) and bool(torch.isnan(got[6, 0, 95]))
    # eps = 0 and a head of zeros: 0 / 0, as the formula has it
    assert bool(torch.isnan(qmv.norm_rope(bad, None, qw, None, pos, f, eps=0.0)[0][3, 1]).all())


def test_gradient_against_differences(qmv):
    """<dx, v> and <dw, v> along random directions against central differences of the f64 forward:
    the truncation is below 1e-7 of the values' size at steps of 1e-3, the bounds above are
    1e-5 of it."""
    T, hq, D, R = 9, 3, 40, 24
    x, w, dy = data((T, hq, D), torch.float32, 21), 1 + data((D,), torch.float32, 22, 0.3), data((T, hq, D), torch.float32, 23)
    pos, f = torch.arange(T) * 100, qmv.rope_freqs(R, device="cpu")
    for layout in ("half", "interleaved"):
        dx, _, dw, _ = qmv.norm_rope_backward(x.cuda(), None, w.cuda(), None, dy.cuda(), None, pos.cuda(), f.cuda(),
                                              layout=layout, amplitude=1.25, weight_offset=0.5)

        def loss(x64, w64):
            return (forward64(x64, w64 + 0.5, pos, f, layout, 1.25, 1e-6)[0] * dy.double()).sum()

        for seed in range(4):
            v, h = data((T, hq, D), torch.float64, 30 + seed), 1e-3
            d = (loss(x.double() + h * v, w.double()) - loss(x.double() - h * v, w.double())) / (2 * h)
            assert abs(float((dx.double().cpu() * v).sum() - d)) <= 1e-5 * float((dx.double().cpu() * v).abs().sum())
            u = data((D,), torch.float64, 40 + seed)
            d = (loss(x.double(), w.double() + h * u) - loss(x.double(), w.double() - h * u)) / (2 * h)
            assert abs(float((dw.double().cpu() * u).sum() - d)) <= 1e-5 * float((dw.double().cpu() * u).abs().sum())


def test_repeats_streams_and_graph(qmv):
    """Calls repeat bit for bit, on another stream too, and a captured pair of calls replays on new inputs."""
    q, k, qw, kw, dq, dk, pos, f = setup(qmv, T=700)
    ref, back = qmv.norm_rope(q, k, qw, kw, pos, f), qmv.norm_rope_backward(q, k, qw, kw, dq, dk, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = qmv.norm_rope(q, k, qw, kw, pos, f, stream=side)
    b = qmv.norm_rope_backward(q, k, qw, kw, dq, dk, pos, f, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a + b, ref + back))
    q2, k2, g2, h2 = (torch.zeros_like(t) for t in (q, k, dq, dk))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = qmv.norm_rope(q2, k2, qw, kw, pos, f) + qmv.norm_rope_backward(q2, k2, qw, kw, g2, h2, pos, f)
    for turn in range(4):
        for t, s in ((q2, q), (k2, k), (g2, dq), (h2, dk)):
            t.copy_(s * (turn + 1))
        graph.replay()
        eager = qmv.norm_rope(q2, k2, qw, kw, pos, f) + qmv.norm_rope_backward(q2, k2, qw, kw, g2, h2, pos, f)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(c, eager))


def test_own_outputs_count_as_changed_and_gradients_are_refused(qmv):
    q, k, qw, kw, dq, dk, pos, f = setup(qmv)
    out = torch.empty_like(q)
    version = out._version
    qmv.norm_rope(q, k, qw, kw, pos, f, q_out=out)
    assert out._version > version
    version = dq._version
    qmv.norm_rope_backward(q, k, qw, kw, dq, dk, pos, f, dq=dq)
    assert dq._version > version
    with pytest.raises(ValueError, match="norm_rope records no gradient"):
        qmv.norm_rope(q, k, qw.clone().requires_grad_(), kw, pos, f)
    with pytest.raises(ValueError, match="norm_rope_backward records no gradient"):
        qmv.norm_rope_backward(q.clone().requires_grad_(), k, qw, kw, dq, dk, pos, f)


def test_more_than_2_31_values(qmv):
    T, hq, D, dt = 70000, 240, 128, torch.bfloat16  # 2.15e9 values
    q = torch.randn((1000, hq, D), dtype=dt, device="cuda").repeat(70, 1, 1)
    pos, f = torch.arange(T, device="cuda"), qmv.rope_freqs(D)
    w = torch.ones(D, dtype=dt, device="cuda")
    say("norm_rope of", q.numel(), "values")
    y, _ = qmv.norm_rope(q, None, w, None, pos, f)
    rows = torch.tensor([0, 1, 999, 34567, 69999])
    check_forward("q", y[rows.cuda()].cpu(), q[rows.cuda()].cpu(), w.cpu(), 0.0, rows, f.cpu(), "half", 1.0, 1e-6)
    back, _, dw, _ = qmv.norm_rope_backward(q, None, w, None, y, None, pos, f)
    g = y[rows.cuda()].cpu()
    check_backward("q", back[rows.cuda()].cpu(), None, q[rows.cuda()].cpu(), g, None, 0.0, rows, f.cpu(), "half", 1.0, 1e-6, 0)
    assert bool(torch.isfinite(dw.float()).all())
