"""The gated feed-forward products and the rotary positions: their measured cases.

Three operators that a decoder with block-quantized weights needs around its
projections when it takes many tokens at once (a prompt, a training batch):

  glu      H = act(X Wg^T) * (X Wu^T) over two packed matrices, act one of
           silu, gelu_tanh, gelu; for training also G = X Wg^T and U = X Wu^T
  glu_bwd  from G, U and dH: dG = dH * U * act'(G), dU = dH * act(G) and
           dX = dG Wg + dU Wu (the packed weights are frozen: they get no
           gradient; dG and dU are what trainable adapters beside them need)
  rope     rotary positions of the q and k heads of T tokens at given positions,
           half or interleaved pairs, the first R of D values of each head,
           from per-pair frequencies; inverse = the gradient

The matrix cores take both operands in the activations' 16-bit type, so a
weight enters the products as W~ = its dequantized value rounded once to that
type (the value a 16-bit model holds); that is part of the operators'
definition and of both reference forms here.

The weights are handed over in the library's packed layout (include/qmv.h,
"Packed layout, version 1"), as a program keeps them; the plain form reads the
same bytes.
"""
import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------ packed formats

FORMATS = ("q8_0", "w4a16_g64", "q4k", "q6k", "q4_0", "q5_0", "q5k", "bf16", "i8row")
BLOCK = {"q8_0": 32, "w4a16_g64": 64, "q4k": 256, "q6k": 256, "q4_0": 32, "q5_0": 32, "q5k": 256, "bf16": 32,
         "i8row": 32}


def _planes(fmt, N, K):
    """Bytes of each plane; every plane starts at a multiple of 256 bytes."""
    return {
        "q8_0": [N * K, N * K // 16],
        "w4a16_g64": [N * K // 2, N * K // 16],
        "q4k": [N * K // 2, N * K // 16],
        "q6k": [N * K // 2, N * K // 4, N * K // 16, N * K // 128],
        "q4_0": [N * K // 2, N * K // 16],
        "q5_0": [N * K // 2, N * K // 8, N * K // 16],
        "q5k": [N * K // 2, N * K // 8, N * K // 16],
        "bf16": [2 * N * K],
        "i8row": [N * K, 4 * N],
    }[fmt]


def _offsets(fmt, N, K):
    offs, at = [], 0
    for b in _planes(fmt, N, K):
        offs.append(at)
        at += (b + 255) // 256 * 256
    return offs, at


def _random_packed(fmt, N, K, gen):
    """A packed matrix of random codes whose weights have mean about 0 and
    standard deviation about 1 / sqrt(K), as trained projections have."""
    dev = gen.device
    sizes = _planes(fmt, N, K)
    offs, total = _offsets(fmt, N, K)
    W = torch.randint(0, 256, (total,), dtype=torch.uint8, device=dev, generator=gen)  # the codes
    sigma = 1.0 / math.sqrt(K)

    def put(i, t):
        b = t.contiguous().view(torch.uint8).reshape(-1)
        W[offs[i]:offs[i] + sizes[i]] = b

    def spread(shape, mid):  # block scales between half and one and a half times their middle
        return (mid * (0.5 + torch.rand(shape, device=dev, generator=gen)))

    if fmt == "q8_0":
        put(1, spread((N, K // 32), sigma / 74).half())
    elif fmt == "w4a16_g64":
        s = spread((N, K // 64), sigma / 4.6).half()
        z = (6 + 3 * torch.rand((N, K // 64), device=dev, generator=gen)).half()
        put(1, torch.stack([s, z], -1))
    elif fmt in ("q4k", "q5k"):
        mid = 7.5 if fmt == "q4k" else 15.5
        d = spread((N, K // 256), sigma / (27 * mid)).half()
        dmin = (mid * d.float() * (0.9 + 0.2 * torch.rand(d.shape, device=dev, generator=gen))).half()
        rec = torch.randint(0, 256, (N, K // 256, 16), dtype=torch.uint8, device=dev, generator=gen)
        rec[..., 0:2] = d.unsqueeze(-1).view(torch.uint8)
        rec[..., 2:4] = dmin.unsqueeze(-1).view(torch.uint8)
        put(1 if fmt == "q4k" else 2, rec)
    elif fmt == "q6k":
        put(2, torch.randint(-64, 64, (N, K // 16), dtype=torch.int8, device=dev, generator=gen))
        put(3, spread((N, K // 256), sigma / 680).half())
    elif fmt == "q4_0":
        put(1, spread((N, K // 32), sigma / 4.6).half())
    elif fmt == "q5_0":
        put(2, spread((N, K // 32), sigma / 9.2).half())
    elif fmt == "bf16":
        put(0, (sigma * torch.randn((N, K), device=dev, generator=gen)).bfloat16())
    else:
        put(1, spread((N,), sigma / 74).float())
    return W


def _dequant(fmt, W, N, K):
    """The weights of a packed matrix, in f32 (plain form)."""
    sizes = _planes(fmt, N, K)
    offs, _ = _offsets(fmt, N, K)
    p = [W[o:o + b] for o, b in zip(offs, sizes)]

    def f16(t, *shape):
        return t.view(torch.float16).reshape(*shape).float()

    def nibbles():
        b = p[0].view(N, K // 2)
        return torch.stack([b & 15, b >> 4], -1).view(N, K)

    def fifth():  # bit 4 of weight 8i + 2c + e of a 32-weight unit is bit 8c + 2i + e of its word
        k = torch.arange(32, device=W.device)
        sh = 8 * ((k % 8) // 2) + 2 * (k // 8) + k % 2
        w = p[1].view(torch.int32).view(N, K // 32, 1)
        return (((w >> sh) & 1) << 4).view(N, K)

    def superblocks(t):  # d, dmin [N][K/256] and the 6-bit sc, m [N][K/32]
        b = t.view(N, K // 256, 16)
        d, dmin = f16(b[..., 0:2].contiguous(), N, K // 256), f16(b[..., 2:4].contiguous(), N, K // 256)
        v = b[..., 4:16].long()
        w8 = torch.arange(6, device=W.device) * 8
        lo = (v[..., 0:6] << w8).sum(-1, keepdim=True)
        hi = (v[..., 6:12] << w8).sum(-1, keepdim=True)
        s6 = torch.arange(8, device=W.device) * 6
        sc, m = ((lo >> s6) & 63).float(), ((hi >> s6) & 63).float()
        return (d.unsqueeze(-1) * sc).view(N, K // 32, 1), (dmin.unsqueeze(-1) * m).view(N, K // 32, 1)

    if fmt == "q8_0":
        w = f16(p[1], N, K // 32, 1) * p[0].view(torch.int8).view(N, K // 32, 32).float()
    elif fmt == "w4a16_g64":
        sz = f16(p[1], N, K // 64, 2)
        w = sz[..., 0:1] * (nibbles().view(N, K // 64, 64).float() - sz[..., 1:2])
    elif fmt == "q4k":
        ds, dm = superblocks(p[1])
        w = ds * nibbles().view(N, K // 32, 32).float() - dm
    elif fmt == "q5k":
        ds, dm = superblocks(p[2])
        w = ds * (nibbles().int() | fifth()).view(N, K // 32, 32).float() - dm
    elif fmt == "q6k":
        k = torch.arange(16, device=W.device)
        sh = 8 * ((k % 8) // 2) + 2 * (2 * (k // 8) + k % 2)
        hi = (p[1].view(torch.int32).view(N, K // 16, 1) >> sh) & 3
        q = nibbles().view(N, K // 16, 16).int() | (hi << 4)
        ds = f16(p[3], N, K // 256, 1) * p[2].view(torch.int8).view(N, K // 256, 16).float()
        w = ds.view(N, K // 16, 1) * (q.float() - 32)
    elif fmt == "q4_0":
        w = f16(p[1], N, K // 32, 1) * (nibbles().view(N, K // 32, 32).float() - 8)
    elif fmt == "q5_0":
        w = f16(p[2], N, K // 32, 1) * ((nibbles().int() | fifth()).view(N, K // 32, 32).float() - 16)
    elif fmt == "bf16":
        w = p[0].view(torch.bfloat16).float()
    else:
        w = p[1].view(torch.float32).view(N, 1) * p[0].view(torch.int8).view(N, K).float()
    return w.reshape(N, K)


# -------------------------------------------------------------------- cases

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token through a gated block that a GeGLU model holds in 16-bit arithmetic: launch latency and weight stream
        dict(name="glu 1 token", op="glu", fmt="w4a16_g64", M=1, N=5632, K=2048, act="gelu_tanh", dtype="bf16", save=False),
        # a short chat turn on the 1.1B decoder's MLP
        dict(name="glu 16 tokens q4k", op="glu", fmt="q4k", M=16, N=5632, K=2048, act="silu", dtype="bf16", save=False),
        # a ragged prompt over a small odd-sized block, fp16
        dict(name="glu 197 tokens q6k odd", op="glu", fmt="q6k", M=197, N=1333, K=768, act="gelu", dtype="f16", save=False),
        # a prompt of the 1.1B decoder
        dict(name="glu 512 tokens", op="glu", fmt="w4a16_g64", M=512, N=5632, K=2048, act="silu", dtype="bf16", save=False),
        # forward of a training batch: G and U are kept for the backward pass
        dict(name="glu 8192 tokens training", op="glu", fmt="w4a16_g64", M=8192, N=5632, K=2048, act="silu", dtype="bf16",
             save=True),
        # backward of a handful of tokens (preference tuning of a short answer), dense weights
        dict(name="glu_bwd 24 tokens", op="glu_bwd", fmt="bf16", M=24, N=5632, K=2048, act="silu", dtype="bf16"),
        # backward of one ragged sequence, odd feed-forward width
        dict(name="glu_bwd 391 tokens odd", op="glu_bwd", fmt="q4k", M=391, N=2731, K=1024, act="gelu_tanh", dtype="f16"),
        # backward of the training batch
        dict(name="glu_bwd 8192 tokens", op="glu_bwd", fmt="w4a16_g64", M=8192, N=5632, K=2048, act="silu", dtype="bf16"),
        # the q and k heads of one decoded token, as the matvec writes them (f32)
        dict(name="rope 1 token", op="rope", T=1, q_heads=32, k_heads=4, D=64, R=64, layout="half", dtype="f32",
             inverse=False, fused=False, far=2048),
        # a prompt, heads taken out of one fused q/k/v product (strided)
        dict(name="rope 4096 tokens fused qkv", op="rope", T=4096, q_heads=32, k_heads=4, D=64, R=64, layout="half",
             dtype="bf16", inverse=False, fused=True, far=4096),
        # far positions of a long context, part of the head, interleaved pairs
        dict(name="rope 32768 tokens far part", op="rope", T=32768, q_heads=16, k_heads=8, D=128, R=96,
             layout="interleaved", dtype="f16", inverse=False, fused=False, far=1000000),
        # gradient of a training batch's q and k
        dict(name="rope 8191 tokens inverse", op="rope", T=8191, q_heads=32, k_heads=4, D=64, R=64, layout="half",
             dtype="bf16", inverse=True, fused=False, far=8192),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("glu", "glu", "glu_bwd", "glu_bwd", "rope"))
    if op == "rope":
        D = 2 * rng.randint(16, 128)
        layout = rng.choice(("half", "interleaved"))
        R = D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        hq = rng.randint(1, 40)
        hk = rng.choice((0, 1, hq, rng.randint(1, 8)))
        T = min(_log(rng, 1, 32768), max(1, 32768 * 24 * 128 // ((hq + hk) * D)))
        return dict(op=op, T=T, q_heads=hq, k_heads=hk, D=D, R=R, layout=layout, dtype=rng.choice(("f32", "bf16", "f16")),
                    inverse=rng.random() < 0.4, fused=rng.random() < 0.5, far=_log(rng, max(T, 64), 2000000))
    fmt = rng.choice(FORMATS)
    M = _log(rng, 1, 8192)
    N = _log(rng, 32, 5632)
    if rng.random() < 0.6:
        N = max(32, N // 64 * 64)
    b = BLOCK[fmt]
    K = _log(rng, 64, 4096) // b * b or b
    if M * N * K > 8192 * 5632 * 2048:
        K = max(b, 8192 * 5632 * 2048 // (M * N) // b * b)
    c = dict(op=op, fmt=fmt, M=M, N=N, K=K, act=rng.choice(("silu", "gelu_tanh", "gelu")), dtype=rng.choice(("bf16", "f16")))
    if op == "glu":
        c["save"] = rng.random() < 0.5
    return c


# -------------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(shape, device="cuda", generator=gen)).to(DT[c["dtype"]])

    if c["op"] == "rope":
        T, hq, hk, D, R = (c[k] for k in ("T", "q_heads", "k_heads", "D", "R"))
        if c["fused"]:  # q, k and v of a token side by side
            qkv = randn(T, hq + 2 * hk, D)
            c["q"], c["k"] = qkv[:, :hq], qkv[:, hq:hq + hk] if hk else None
        else:
            c["q"], c["k"] = randn(T, hq, D), randn(T, hk, D) if hk else None
        # packed sequences: each starts anew at some position of the range
        start = torch.randint(0, c["far"], (1,), device="cuda", generator=gen)
        c["pos"] = (start + torch.arange(T, device="cuda")) % c["far"]
        # frequencies stretched for a long context: the slow pairs are interpolated by 4, the fast ones kept, a ramp between
        i = torch.arange(R // 2, dtype=torch.float64)
        f = 10000.0 ** (-2 * i / R)
        keep = ((f * c["far"] / (2 * math.pi) - 1) / 31).clamp(0, 1)
        c["freqs"] = (f * keep + f / 4 * (1 - keep)).float().cuda()
        c["amplitude"] = 0.1 * math.log(4.0) + 1.0
        return c
    M, N, K = c["M"], c["N"], c["K"]
    c["Wg"] = _random_packed(c["fmt"], N, K, gen)
    c["Wu"] = _random_packed(c["fmt"], N, K, gen)
    if c["op"] == "glu":
        c["X"] = randn(M, K)
    else:
        c["G"], c["U"], c["dH"] = randn(M, N), randn(M, N), randn(M, N, scale=0.01)
    return c


# -------------------------------------------------------------------- a pass


def _act(name, g):
    """act(g) and act'(g)."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    p = 0.5 * torch.erfc(-g * math.sqrt(0.5))
    return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _rotate(x, cos, sin, R, layout):
    """Rotary pairs of x [T][heads][D] (f32) by cos, sin [T][R/2]."""
    c, s = cos[:, None, :], sin[:, None, :]
    y = x.clone()
    if layout == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * c - b * s, b * c + a * s
    return y


def _run_own(c):
    import gemm_dequant_matvec_amd as qmv

    if c["op"] == "rope":
        q, k = qmv.rope(c["q"], c["k"], c["pos"], c["freqs"], layout=c["layout"], amplitude=c["amplitude"],
                        inverse=c["inverse"])
        return {"q": q, "k": k}
    if c["op"] == "glu":
        if c["save"]:
            H, G, U = qmv.gemm_glu(c["fmt"], c["Wg"], c["Wu"], c["X"], c["N"], c["K"], act=c["act"], save=True)
            return {"H": H, "G": G, "U": U}
        return {"H": qmv.gemm_glu(c["fmt"], c["Wg"], c["Wu"], c["X"], c["N"], c["K"], act=c["act"])}
    # both reference forms sum dX over dG and dU as they are before their rounding
    dX, dG, dU = qmv.gemm_glu_backward(c["fmt"], c["Wg"], c["Wu"], c["G"], c["U"], c["dH"], c["N"], c["K"], act=c["act"],
                                       unrounded=True)
    return {"dX": dX, "dG": dG, "dU": dU}


def run(state):
    if own:
        return _run_own(state)
    c = state
    t = DT[c["dtype"]]
    if c["op"] == "rope":
        a = c["pos"].double()[:, None] * c["freqs"].double()  # far angles need 64 bits
        if c["inverse"]:
            a = -a
        cos, sin = (c["amplitude"] * a.cos()).float(), (c["amplitude"] * a.sin()).float()
        q = _rotate(c["q"].float(), cos, sin, c["R"], c["layout"]).to(t)
        k = None if c["k"] is None else _rotate(c["k"].float(), cos, sin, c["R"], c["layout"]).to(t)
        return {"q": q, "k": k}
    Wg = _dequant(c["fmt"], c["Wg"], c["N"], c["K"]).to(t).float()  # W~, the operand's type
    Wu = _dequant(c["fmt"], c["Wu"], c["N"], c["K"]).to(t).float()
    if c["op"] == "glu":
        x = c["X"].float()
        g, u = x @ Wg.t(), x @ Wu.t()
        h = (_act(c["act"], g)[0] * u).to(t)
        return {"H": h, "G": g.to(t), "U": u.to(t)} if c["save"] else {"H": h}
    g, u, dh = c["G"].float(), c["U"].float(), c["dH"].float()
    a, da = _act(c["act"], g)
    dg, du = dh * u * da, dh * a
    return {"dX": (dg @ Wg + du @ Wu).to(t), "dG": dg.to(t), "dU": du.to(t)}


# ------------------------------------------------------------------ the work


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * (c["q_heads"] + c["k_heads"])
        e = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * n * c["D"] * e + 8 * c["T"] + 2 * c["R"], "flops": 3 * n * c["R"]}
    M, N, K = c["M"], c["N"], c["K"]
    w = 2 * sum(_planes(c["fmt"], N, K))
    mn = 5 if c["op"] == "glu_bwd" else 3 if c["save"] else 1
    return {"bytes": w + 2 * M * K + 2 * mn * M * N, "flops": 4 * M * N * K}


# ------------------------------------------- the definition, in 64 bits, apart


def _exact_weights(fmt, W, N, K, t):
    """W~ in f64 from the packed bytes, block by block as the layout's text has them."""
    raw = W.cpu().numpy()
    offs, _ = _offsets(fmt, N, K)
    sizes = _planes(fmt, N, K)
    plane = [raw[o:o + s] for o, s in zip(offs, sizes)]
    half = lambda i: plane[i].view("<f2").astype(np.float64)  # noqa: E731
    if fmt == "bf16":
        w = (plane[0].view("<u2").astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    elif fmt in ("q8_0", "i8row"):
        q = plane[0].view(np.int8).astype(np.float64)
        w = q * (np.repeat(half(1), 32) if fmt == "q8_0" else np.repeat(plane[1].view("<f4").astype(np.float64), K))
    else:
        q = np.empty(N * K, np.float64)
        q[0::2], q[1::2] = plane[0] % 16, plane[0] // 16
        if fmt in ("q5_0", "q5k"):
            words = plane[1].view("<u4")
            for i in range(4):
                for c in range(4):
                    for e in range(2):
                        q[8 * i + 2 * c + e::32] += 16 * ((words >> np.uint32(8 * c + 2 * i + e)) % 2)
        if fmt == "q6k":
            words = plane[1].view("<u4")
            for c in range(4):
                for f in range(4):
                    q[8 * (f // 2) + 2 * c + f % 2::16] += 16 * ((words >> np.uint32(8 * c + 2 * f)) % 4)
            w = np.repeat(np.repeat(half(3), 16) * plane[2].view(np.int8), 16) * (q - 32)
        elif fmt in ("q4k", "q5k"):
            rec = plane[-1].reshape(-1, 16)
            d, dmin = (rec[:, j:j + 2].copy().view("<f2").astype(np.float64) for j in (0, 2))
            bits = np.unpackbits(rec[:, 4:], axis=1, bitorder="little").reshape(-1, 16, 6)
            v = (bits * 2 ** np.arange(6)).sum(-1)
            w = np.repeat((d * v[:, :8]).reshape(-1), 32) * q - np.repeat((dmin * v[:, 8:]).reshape(-1), 32)
        elif fmt == "w4a16_g64":
            sz = half(1)
            w = np.repeat(sz[0::2], 64) * (q - np.repeat(sz[1::2], 64))
        else:
            w = np.repeat(half(len(plane) - 1), 32) * (q - (8 if fmt == "q4_0" else 16))
    return torch.from_numpy(w.reshape(N, K)).to(W.device).to(t).double()


def _exact_act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g), torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    if name == "gelu_tanh":  # (1 + tanh z) / 2 = sigmoid(2 z)
        z2 = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
        s = torch.sigmoid(z2)
        return g * s, s + g * s * torch.sigmoid(-z2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g * g)
    cdf = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
    return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "rope":
        turns = c["pos"].double()[:, None] * c["freqs"].double() * (-1 if c["inverse"] else 1)
        z = torch.polar(torch.full_like(turns, c["amplitude"]), turns)[:, None, :]
        out = {}
        for name in ("q", "k"):
            x = c[name]
            if x is None:
                out[name] = None
                continue
            x, R = x.double(), c["R"]
            shape = (x.shape[0], x.shape[1], 2, R // 2) if c["layout"] == "half" else (x.shape[0], x.shape[1], R // 2, 2)
            ab = x[..., :R].reshape(shape)
            ab = ab.transpose(-1, -2) if c["layout"] == "half" else ab
            r = torch.view_as_real(torch.view_as_complex(ab.contiguous()) * z)
            r = r.transpose(-1, -2) if c["layout"] == "half" else r
            out[name] = torch.cat([r.reshape(x.shape[0], x.shape[1], R), x[..., R:]], -1)
        return out
    t = DT[c["dtype"]]
    Wg, Wu = (_exact_weights(c["fmt"], c[w], c["N"], c["K"], t) for w in ("Wg", "Wu"))
    if c["op"] == "glu":
        x = c["X"].double()
        g, u = torch.mm(x, Wg.t()), torch.mm(x, Wu.t())
        h = _exact_act(c["act"], g)[0] * u
        return {"H": h, "G": g, "U": u} if c["save"] else {"H": h}
    g, u, dh = c["G"].double(), c["U"].double(), c["dH"].double()
    a, da = _exact_act(c["act"], g)
    dg, du = dh * u * da, dh * a
    return {"dX": torch.mm(dg, Wg) + torch.mm(du, Wu), "dG": dg, "dU": du}
