"""The key / value cache in plain tensor operations on the CPU: the layout's text
value by value, the quantisation step by step."""
from __future__ import annotations

import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def set_bytes(fmt, D):
    return D // 32 * (2 * (512 if fmt == "q8_0" else 256) + 64)


def places(fmt, heads, D, page, page_id, token):
    """Byte indexes of one token's K and V codes, and f16 indexes of its K and V scales: [heads][D] and
    [heads][D / 32]."""
    nb, C = D // 32, 512 if fmt == "q8_0" else 256
    rec = page // 16 * set_bytes(fmt, D)
    base = (page_id * heads + torch.arange(heads)) * rec + token // 16 * set_bytes(fmt, D)
    t, d = token % 16, torch.arange(D)
    b, e = d // 32, d % 32
    if fmt == "q8_0":
        k = 512 * b + 8 * (16 * (e // 8) + t) + e % 8
        v = 512 * b + 4 * (2 * (16 * (t // 4) + e % 16) + e // 16) + t % 4
    else:
        k = 256 * b + 4 * (16 * (e // 8) + t) + e % 4
        v = 256 * b + 4 * (16 * (t // 4) + e % 16) + t % 4
    s = 4 * (nb * (t // 4) + torch.arange(nb)) + t % 4
    return (base[:, None] + k, base[:, None] + nb * C + v, (base[:, None] + 2 * nb * C) // 2 + s,
            (base[:, None] + 2 * nb * C + 32 * nb) // 2 + s)


def value(fmt, data, heads, D, page, page_id, token):
    """K and V [heads][D] (f64) of one token; data: the cache's bytes on the CPU."""
    ki, vi, ks, vs = places(fmt, heads, D, page, page_id, token)
    h, e = data.view(torch.float16), torch.arange(D) % 32
    out = []
    for ci, si, high in ((ki, ks, e % 8 >= 4), (vi, vs, e >= 16)):
        q = data[ci].long()
        q = q - 128 if fmt == "q8_0" else torch.where(high, q // 16, q % 16) - 8
        out.append(q.double() * h[si].double().repeat_interleave(32, -1))
    return out


def quantised(fmt, x):
    """(codes, scales) of x [..][D]: the definition's steps, one f32 operation each."""
    s, low, top = (127.0, -127, 127) if fmt == "q8_0" else (7.5, -8, 7)
    x = x.float().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    d = torch.clamp(amax / torch.tensor(s), max=65504.0).half()
    d = torch.where(bad, torch.full_like(d, float("nan")), d)
    inv = torch.where(d > 0, 1 / d.float(), torch.zeros(()))
    q = torch.where(bad, torch.zeros(()), torch.clamp(torch.round(torch.nan_to_num(x) * torch.nan_to_num(inv)), low, top))
    return q.flatten(-2).long(), d.squeeze(-1)


def stands_for(fmt, x):
    """What the cache holds of x, in f64 (exact)."""
    q, d = quantised(fmt, x)
    return q.double() * d.double().repeat_interleave(32, -1)


def half_step(dt):
    return torch.finfo(dt).eps / 2, 2.0 ** -25 if dt == torch.float16 else 0.0

