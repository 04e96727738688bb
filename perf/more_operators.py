"""Between a decoder's q / k / v products and its o product: their measured cases.

  norm_rope      the norm of every q and k head and its rotary position in one pass
  norm_rope_bwd  its gradient: dq, dk and the gradients of the two norm weights
  cache_write    the keys and values of new tokens go into a paged cache of 8-bit
                 or 4-bit blocks, and what it now holds of them is read back
  cache_read     whole sequences are read back from such a cache
  attention      queries over the cache: single tokens, prompt chunks, ragged
                 batches, a window, a prefix that the whole batch shares

The cache (formats q8_0 and q4_0: blocks of 32 values of a head, w = d q with an
f16 scale d).  A page holds `page` tokens (a multiple of 16) of every k / v head;
the record of a page and head is a run of records of 16 tokens, each made of four
planes: K codes, V codes (512 bytes per block of 32 dimensions, q4_0: 256), K
scales, V scales (32 bytes per block).  With token t, block b, dimension 32 b + e
and nb blocks a head:
  K, q8_0  byte 512 b + 8 (16 (e / 8) + t) + e % 8              holds q + 128
  K, q4_0  byte 256 b + 4 (16 (e / 8) + t) + e % 4              holds q + 8 in its low (e % 8 < 4) or high half
  V, q8_0  byte 512 b + 4 (2 (16 (t / 4) + e % 16) + e / 16) + t % 4  holds q + 128
  V, q4_0  byte 256 b + 4 (16 (t / 4) + e % 16) + t % 4         holds q + 8 in its low (e < 16) or high half
  scales   f16 number 4 (nb (t / 4) + b) + t % 4
Position p of sequence b is token p % page of page table[b][p / page].

A batch: tokens q_start[b] .. q_start[b + 1] - 1 are the last ones of sequence b, which
is kv_len[b] long with them.

Quantising a block: d = f16(min(max |x| / s, 65504)), s = 127 (q8_0) or 7.5 (q4_0),
q = round-half-even(x * (1 / d)) clamped to -127 .. 127 or -8 .. 7, q = 0 where d = 0,
each step one f32 operation.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # the q and k heads of one decoded token, out of the matvec's f32 rows: latency
        dict(name="norm rope 1 token", op="norm_rope", T=1, q_heads=32, k_heads=4, D=64, R=64, layout="half", dtype="f32",
             w_dtype="f32", offset=0.0, fused=True),
        # a prompt or the forward of a training batch, heads taken out of one fused product
        dict(name="norm rope 16384 tokens fused qkv", op="norm_rope", T=16384, q_heads=32, k_heads=8, D=128, R=128,
             layout="half", dtype="bf16", w_dtype="bf16", offset=0.0, fused=True),
        # gradient of one short ragged answer, an odd head, part of it turned, weights stored as w - 1
        dict(name="norm rope backward 61 tokens odd", op="norm_rope_bwd", T=61, q_heads=12, k_heads=3, D=80, R=48,
             layout="interleaved", dtype="f16", w_dtype="f32", offset=1.0, fused=False),
        # gradient of the training batch
        dict(name="norm rope backward 16384 tokens", op="norm_rope_bwd", T=16384, q_heads=32, k_heads=8, D=128, R=128,
             layout="half", dtype="bf16", w_dtype="bf16", offset=0.0, fused=True),
        # one decode step of a batch: a token for each of 48 sequences
        dict(name="cache write 48 tokens q8_0", op="cache_write", fmt="q8_0", B=48, heads=4, D=64, page=16, dtype="f32",
             long=2000, new=1, mix=1),
        # a batch of ragged prompts
        dict(name="cache write ragged prompts q4_0", op="cache_write", fmt="q4_0", B=8, heads=8, D=128, page=64, dtype="bf16",
             long=500, new=8000, mix=2),
        # one short conversation, odd length, f32 for inspection or a host copy
        dict(name="cache read 777 tokens q4_0", op="cache_read", fmt="q4_0", B=1, heads=2, D=96, page=48, dtype="f32",
             long=777, new=777, mix=0),
        # many long sequences, for dense attention or to move them elsewhere
        dict(name="cache read ragged sequences q8_0", op="cache_read", fmt="q8_0", B=24, heads=8, D=128, page=64, dtype="bf16",
             long=16000, new=16000, mix=4),
        # one decoded token of the 1.1B decoder
        dict(name="attention 1 token", op="attention", fmt="q8_0", B=1, heads=4, group=8, D=64, page=16, dtype="f32",
             long=2048, new=1, window=0, prefix=0, mix=0),
        # a decode step of a ragged batch of long sequences
        dict(name="attention 64 ragged sequences", op="attention", fmt="q8_0", B=64, heads=8, group=4, D=128, page=64,
             dtype="bf16", long=16000, new=1, window=0, prefix=0, mix=6),
        # a decode step of many requests behind one long shared instruction
        dict(name="attention shared prefix", op="attention", fmt="q4_0", B=96, heads=8, group=4, D=128, page=64, dtype="f16",
             long=1000, new=1, window=0, prefix=8200, mix=7),
        # chunks of prompts, odd head counts and lengths, a sliding window
        dict(name="attention prompt chunks window", op="attention", fmt="q8_0", B=3, heads=2, group=7, D=96, page=32,
             dtype="bf16", long=6000, new=700, window=1500, prefix=0, mix=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "norm_rope_bwd", "cache_write", "cache_read", "attention", "attention"))
    if op.startswith("norm_rope"):
        D = rng.randint(16, 256)
        layout = rng.choice(("half", "interleaved"))
        R = D // 2 * 2 if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        hq = rng.randint(1, 40)
        hk = rng.choice((0, 1, hq, rng.randint(1, 8)))
        T = min(_log(rng, 1, 16384), max(1, 16384 * 40 * 128 // ((hq + hk) * D)))
        dtype = rng.choice(("f32", "bf16", "f16"))
        if dtype == "f32":
            T = (T + 1) // 2
        return dict(op=op, T=T, q_heads=hq, k_heads=hk, D=D, R=R, layout=layout, dtype=dtype,
                    w_dtype=rng.choice((dtype, "f32")), offset=float(rng.choice((0, 0, 1))), fused=rng.random() < 0.5)
    fmt = rng.choice(("q8_0", "q4_0"))
    D = 32 * rng.randint(1, 8)
    heads = rng.randint(1, 8)
    page = 16 * rng.choice((1, 2, 3, 4, 8, 16))
    dtype = rng.choice(("f32", "bf16", "f16"))
    B = _log(rng, 1, 64)
    c = dict(op=op, fmt=fmt, B=B, heads=heads, D=D, page=page, dtype=dtype, mix=rng.randint(0, 10 ** 6))
    most = 2 ** 26 // (B * heads * D)  # tokens a sequence
    if op == "cache_write":
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(8000, most // 2)))
        c["long"] = _log(rng, 1, max(1, min(4000, most)))
    elif op == "cache_read":
        c["long"] = c["new"] = _log(rng, 1, max(1, min(16000, most)))
    else:
        c["group"] = rng.randint(1, 16)
        c["long"] = _log(rng, 1, max(1, min(16000, most)))
        c["new"] = 1 if rng.random() < 0.6 else _log(rng, 1, 700)
        c["prefix"] = _log(rng, 16, 8200) if rng.random() < 0.35 else 0
        c["window"] = _log(rng, 1, 2 * c["long"]) if rng.random() < 0.3 else 0
        # no more scores than the largest listed case has
        while B * heads * c["group"] * c["new"] * (c["long"] + c["prefix"] + c["new"]) * D > 4 * 10 ** 10:
            c["new"], c["prefix"], c["long"] = (c["new"] + 1) // 2, c["prefix"] // 2, (c["long"] + 1) // 2
    return c


def _batch(c):
    """(tokens of the call, length with them) of each sequence: ragged where there are several of many tokens, with
    empty, one-token and longest ones among them."""
    rng = random.Random(c["mix"])
    out = []
    for b in range(c["B"]):
        old, new = c["long"], c["new"]
        if b:  # the first is the longest
            old = rng.choice((0, 1, old, rng.randint(0, old), rng.randint(0, old), rng.randint(old // 2, old)))
            new = new if new == 1 else rng.choice((0, 1, new, rng.randint(0, new), rng.randint(new // 2, new)))
        if c["op"] == "cache_read":
            out.append((old, old))
        else:
            p = c.get("prefix", 0)
            out.append((new, p + max(old, new) if c["op"] == "attention" else old + new))
    return out


# ------------------------------------------------------------ the cache's bytes


def _sizes(c):
    """(blocks a head, bytes of codes a block of 16 tokens, bytes of a 16-token record, bytes of a page's head)."""
    nb, code = c["D"] // 32, 512 if c["fmt"] == "q8_0" else 256
    sub = nb * (2 * code + 64)
    return nb, code, sub, c["page"] // 16 * sub


def _unpack(c, pages):
    """K and V [n * page][heads][D] (f32) of n pages of bytes."""
    nb, code, sub, rec = _sizes(c)
    n, H = pages.shape[0], c["heads"]
    r = pages.view(n * H * (c["page"] // 16), sub)
    m = r.shape[0]
    k, v = r[:, :nb * code], r[:, nb * code:2 * nb * code]
    if c["fmt"] == "q8_0":
        k = k.reshape(m, nb, 4, 16, 8).float() - 128
        v = v.reshape(m, nb, 4, 16, 2, 4).float() - 128
    else:
        k = k.reshape(m, nb, 4, 16, 1, 4)
        k = torch.cat([k & 15, k >> 4], 4).reshape(m, nb, 4, 16, 8).float() - 8
        v = v.reshape(m, nb, 4, 16, 1, 4)
        v = torch.cat([v & 15, v >> 4], 4).float() - 8
    k = k.permute(0, 3, 1, 2, 4).reshape(m, 16, nb, 32)  # record, token, block, dimension
    v = v.permute(0, 2, 5, 1, 4, 3).reshape(m, 16, nb, 32)
    s = r[:, 2 * nb * code:].contiguous().view(torch.float16).view(m, 2, 4, nb, 4).permute(1, 0, 2, 4, 3).reshape(2, m, 16, nb, 1)
    s = s.float()

    def by_token(x):
        x = x.reshape(n, H, c["page"], c["D"])
        return x.transpose(1, 2).reshape(n * c["page"], H, c["D"])

    return by_token(k * s[0]), by_token(v * s[1])


def _places(c, table, first, count):
    """The page's head 0 record and token in it of positions first .. first + count - 1 of a table's row."""
    p = torch.arange(first, first + count, device=table.device)
    return table.long()[p // c["page"]], p % c["page"]


def _indices(c, page, tok):
    """For tokens at (page, tok): indexes of the K and V code bytes [t][heads][D] and of the K and V scales (in f16
    numbers) [t][heads][nb]."""
    nb, code, sub, rec = _sizes(c)
    H, dev = c["heads"], page.device
    base = (page[:, None] * H + torch.arange(H, device=dev)) * rec + (tok // 16 * sub)[:, None]
    t = (tok % 16)[:, None, None]
    d = torch.arange(c["D"], device=dev)
    b, e = d // 32, d % 32
    if c["fmt"] == "q8_0":
        k = 512 * b + 8 * (16 * (e // 8) + t) + e % 8
        v = 512 * b + 4 * (2 * (16 * (t // 4) + e % 16) + e // 16) + t % 4
    else:
        k = 256 * b + 4 * (16 * (e // 8) + t) + e % 4
        v = 256 * b + 4 * (16 * (t // 4) + e % 16) + t % 4
    s = 4 * (nb * (t // 4) + torch.arange(nb, device=dev)) + t % 4
    at = base[:, :, None]
    ks = (at + 2 * nb * code) // 2 + s
    return at + k, at + nb * code + v, ks, ks + 16 * nb


# -------------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    dt = DT[c["dtype"]]

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(shape, device="cuda", generator=gen)).to(dt)

    D = c["D"]
    if c["op"].startswith("norm_rope"):
        T, hq, hk, R = (c[k] for k in ("T", "q_heads", "k_heads", "R"))
        if c["fused"]:  # q, k and v of a token side by side
            qkv = randn(T, hq + 2 * hk, D)
            c["q"], c["k"] = qkv[:, :hq], qkv[:, hq:hq + hk] if hk else None
        else:
            c["q"], c["k"] = randn(T, hq, D), randn(T, hk, D) if hk else None
        for w in ("qw", "kw"):  # learned weights, about 1, stored less the offset
            x = 1 - c["offset"] + 0.25 * torch.randn(D, device="cuda", generator=gen)
            c[w] = x.to(DT[c["w_dtype"]]) if w == "qw" or hk else None
        start = torch.randint(0, 4096, (1,), device="cuda", generator=gen)
        c["pos"] = (start + torch.arange(T, device="cuda")) % 4096  # packed sequences
        c["freqs"] = (10000.0 ** (-2 * torch.arange(R // 2, dtype=torch.float64) / R)).float().cuda()
        if c["op"] == "norm_rope_bwd":
            c["dq"], c["dk"] = randn(T, hq, D, scale=0.01), randn(T, hk, D, scale=0.01) if hk else None
        return c

    c["batch"] = _batch(c)
    longest = max(n for _, n in c["batch"])
    width = max(1, -(-longest // c["page"]))
    shared = c.get("prefix", 0) // c["page"]  # whole pages that all sequences have in common
    pages = shared + c["B"] * (width - shared) + 3
    nb, code, sub, rec = _sizes(c)
    order = torch.randperm(pages, device="cuda", generator=gen).int()
    table = order[shared + torch.arange(c["B"], device="cuda")[:, None] * (width - shared)
                  + torch.arange(width, device="cuda") - shared]
    table[:, :shared] = order[:shared]
    c["table"] = table.contiguous()
    starts, lens, at = [0], [], 0
    for new, n in c["batch"]:
        at += new
        starts.append(at)
        lens.append(n)
    c["T"] = at
    c["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    c["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c["max_q"], c["max_kv"] = max(n for n, _ in c["batch"]), longest
    # codes and scales as quantised heads have them: values about N(0, 1)
    m = pages * c["heads"] * (c["page"] // 16)
    data = torch.empty((m, sub), dtype=torch.uint8, device="cuda")
    codes = 2 * nb * code
    step = max(1, 2 ** 27 // sub)
    for i in range(0, m, step):
        z = torch.randn((min(step, m - i), codes), device="cuda", generator=gen)
        if c["fmt"] == "q8_0":
            data[i:i + step, :codes] = (z * 45).round_().clamp_(-127, 127).add_(128).byte()
        else:
            hi = torch.randn(z.shape, device="cuda", generator=gen)
            lo, hi = ((x * 3).round_().clamp_(-8, 7).add_(8).byte() for x in (z, hi))
            data[i:i + step, :codes] = lo | (hi << 4)
    s = (0.5 + torch.rand((m, 32 * nb), device="cuda", generator=gen)) / (45 if c["fmt"] == "q8_0" else 3)
    data[:, codes:] = s.half().view(torch.uint8)
    c["data"], c["pages"] = data.view(pages, c["heads"], rec), pages
    if shared * c["page"] < c.get("prefix", 0):  # the page in which the prefix ends: a copy for each sequence
        own_page = table[:, shared].long()
        c["data"][own_page[1:]] = c["data"][own_page[0]].clone()
    H = c["heads"]
    if c["op"] == "cache_write":
        loud = 1 + 7 * (torch.rand((H, D), device="cuda", generator=gen) < 0.03)  # keys have loud dimensions
        c["k"], c["v"] = randn(at, H, D) * loud.to(dt), randn(at, H, D)
    elif c["op"] == "attention":
        c["q"] = randn(at, H * c["group"], D, scale=2.0)
        c["scale"] = D ** -0.5
    return c


# -------------------------------------------------------------------- a pass


def _run_own(c):
    import gemm_dequant_matvec_amd as qmv

    if c["op"] == "norm_rope":
        q, k = qmv.norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["pos"], c["freqs"], eps=1e-6, layout=c["layout"],
                             weight_offset=c["offset"])
        return {"q": q, "k": k}
    if c["op"] == "norm_rope_bwd":
        dq, dk, dqw, dkw = qmv.norm_rope_backward(c["q"], c["k"], c["qw"], c["kw"], c["dq"], c["dk"], c["pos"], c["freqs"],
                                                  eps=1e-6, layout=c["layout"], weight_offset=c["offset"])
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    cache = qmv.KVCache(c["fmt"], c["pages"], c["heads"], c["D"], c["page"], data=c["data"])
    if c["op"] == "attention":
        return qmv.kv_attention(cache, c["q"], c["table"], c["q_start"], c["kv_len"], scale=c["scale"], window=c["window"],
                                prefix=c["prefix"], max_q=c["max_q"], max_kv=c["max_kv"])
    if c["op"] == "cache_write":
        qmv.kv_write(cache, c["k"], c["v"], c["table"], c["q_start"], c["kv_len"])
    k, v = qmv.kv_read(cache, c["table"], c["q_start"], c["kv_len"], c["T"], dtype=DT[c["dtype"]])
    return {"k": k, "v": v}


def _turn(x, cos, sin, R, layout):
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


def _plain_norm_rope(c):
    t, D = DT[c["dtype"]], c["D"]
    a = c["pos"].double()[:, None] * c["freqs"].double()
    cos, sin = a.cos().float(), a.sin().float()
    out = {}
    for name in ("q", "k"):
        x = c[name]
        if x is None:
            out.update({name: None} if c["op"] == "norm_rope" else {"d" + name: None, "d" + name + "w": None})
            continue
        x, w = x.float(), c[name + "w"].float() + c["offset"]
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6)
        n = x * r
        if c["op"] == "norm_rope":
            out[name] = _turn(n * w, cos, sin, c["R"], c["layout"]).to(t)
            continue
        g = _turn(c["d" + name].float(), cos, -sin, c["R"], c["layout"])
        h = g * w
        out["d" + name] = (r * (h - n * ((h * n).sum(-1, keepdim=True) / D))).to(t)
        out["d" + name + "w"] = (g * n).sum((0, 1)).to(c[name + "w"].dtype)
    return out


def _plain_write(c):
    low, top, s = (-127, 127, 127.0) if c["fmt"] == "q8_0" else (-8, 7, 7.5)
    s = torch.full((1,), s, device="cuda")  # a tensor: a number's reciprocal would be multiplied by
    flat = c["data"].view(-1)
    halves = flat.view(torch.float16)
    T, H = c["T"], c["heads"]
    start, end = c["q_start"][:-1].long(), c["q_start"][1:].long()
    seq = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), end - start, output_size=T)
    pos = torch.arange(T, device="cuda") + (c["kv_len"].long() - end)[seq]
    ki, vi, ksi, vsi = _indices(c, c["table"].long()[seq, pos // c["page"]], pos % c["page"])
    for x, ci, si, far in ((c["k"], ki, ksi, 4), (c["v"], vi, vsi, 16)):
        x = x.float().reshape(T, H, -1, 32)
        d = (x.abs().amax(-1, keepdim=True) / s).clamp(max=65504).half()
        inv = torch.where(d > 0, 1 / d.float(), torch.zeros_like(d, dtype=torch.float32))
        q = (x * inv).round().clamp(low, top)
        if c["fmt"] == "q8_0":
            flat[ci] = (q + 128).byte().view(T, H, -1)
        else:  # a byte has two values: dimensions 4 apart (K), 16 apart (V)
            q = (q + 8).byte().view(T, H, -1, 2, far)
            flat[ci.view(T, H, -1, 2, far)[:, :, :, 0]] = q[:, :, :, 0] | (q[:, :, :, 1] << 4)
        halves[si] = d.squeeze(-1)


def _plain_read(c):
    ks, vs = [], []
    for b, (new, n) in enumerate(c["batch"]):
        used = c["table"][b, :-(-n // c["page"])].long()
        if new:
            k, v = _unpack(c, c["data"][used])
            ks.append(k[n - new:n].to(DT[c["dtype"]]))
            vs.append(v[n - new:n].to(DT[c["dtype"]]))
    return {"k": torch.cat(ks), "v": torch.cat(vs)}


def _plain_attention(c):
    out, at, H, G, D = [], 0, c["heads"], c["group"], c["D"]
    for b, (new, n) in enumerate(c["batch"]):
        if not new:
            continue
        first = max(0, n - new - c["window"] + 1) // c["page"] if c["window"] else 0  # the first page that is seen
        k, v = _unpack(c, c["data"][c["table"][b, first:-(-n // c["page"])].long()])
        first *= c["page"]
        k, v = (x[:n - first].transpose(0, 1).contiguous() for x in (k, v))  # [heads][tokens][D]
        q = c["q"][at:at + new].float().view(new, H, G, D).permute(1, 2, 0, 3).reshape(H, G * new, D)
        s = torch.bmm(q, k.transpose(1, 2).contiguous()) * c["scale"]
        if new > 1 or c["window"]:
            t = torch.arange(first, n, device=s.device)
            pos = torch.arange(n - new, n, device=s.device).repeat(G)[:, None]
            hidden = t > pos
            if c["window"]:
                hidden = hidden | (t <= pos - c["window"])
            s = torch.where(hidden, float("-inf"), s)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.bmm(p, v) / p.sum(-1, keepdim=True)
        out.append(o.view(H, G, new, D).permute(2, 0, 1, 3).reshape(new, H * G, D).to(DT[c["dtype"]]))
        at += new
    return torch.cat(out)


def run(state):
    if own:
        return _run_own(state)
    c = state
    if c["op"].startswith("norm_rope"):
        return _plain_norm_rope(c)
    if c["op"] == "attention":
        return _plain_attention(c)
    if c["op"] == "cache_write":
        _plain_write(c)
    return _plain_read(c)


# ------------------------------------------------------------------ the work


def work(case):
    c, D = case, case["D"]
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"].startswith("norm_rope"):
        n = c["T"] * (c["q_heads"] + c["k_heads"]) * D
        back = c["op"] == "norm_rope_bwd"
        return {"bytes": (3 if back else 2) * n * e + 8 * c["T"], "flops": (14 if back else 7) * n}
    H, batch = c["heads"], _batch(c)
    value = (1 if c["fmt"] == "q8_0" else 0.5) + 1 / 16  # bytes of a cached value
    new = sum(n for n, _ in batch)
    if c["op"] == "cache_read":
        return {"bytes": int(2 * new * H * D * (e + value)), "flops": 2 * new * H * D}
    if c["op"] == "cache_write":  # k, v in, the cache's blocks out, read back
        return {"bytes": int(2 * new * H * D * (2 * e + 2 * value)), "flops": 8 * new * H * D}
    tokens, scores = 0, 0
    prefix = c["prefix"]
    seen_first = None  # of the prefix
    for n, length in batch:
        if not n:
            continue
        lo = max(0, length - n - c["window"] + 1) if c["window"] else 0
        tokens += length - max(lo, prefix)
        if lo < prefix:
            seen_first = lo if seen_first is None else min(lo, seen_first)
        for i in range(n):
            pos = length - n + i
            scores += min(pos + 1, c["window"]) if c["window"] else pos + 1
    if seen_first is not None:
        tokens += prefix - seen_first
    return {"bytes": int(2 * tokens * H * D * value) + 2 * new * H * c["group"] * D * e, "flops": 4 * scores * H * c["group"] * D}


# ------------------------------------------- the definition, in 64 bits, apart


def _cached(c, b, first, count):
    """K and V [count][heads][D] (f64) of positions first .. of sequence b, value by value from the layout's text."""
    ki, vi, ksi, vsi = _indices(c, *_places(c, c["table"][b], first, count))
    flat = c["data"].view(-1)
    halves = flat.view(torch.float16)
    e = torch.arange(c["D"], device=flat.device) % 32
    out = []
    for ci, si, high in ((ki, ksi, e % 8 >= 4), (vi, vsi, e >= 16)):
        q = flat[ci].double()
        if c["fmt"] == "q8_0":
            q = q - 128
        else:
            q = torch.where(high, torch.floor(q / 16), torch.remainder(q, 16)) - 8
        out.append(q * halves[si].double().repeat_interleave(32, -1))
    return out


def _exact_quantised(c, x):
    """What a block stands for, by the definition's steps: f64 results rounded to f32 (or f16) are the f32 operations'."""
    s, low, top = (127.0, -127, 127) if c["fmt"] == "q8_0" else (7.5, -8, 7)
    s = torch.full((1,), s, dtype=torch.float64, device="cuda")
    x = x.double().unflatten(-1, (-1, 32))
    d = torch.clamp((x.abs().amax(-1, keepdim=True) / s).float(), max=65504.0).half().double()
    inv = torch.where(d > 0, (1 / d).float().double(), 0.0)
    return (torch.clamp(torch.round((x * inv).float().double()), low, top) * d).flatten(-2)


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"].startswith("norm_rope"):
        turns = c["pos"].double()[:, None] * c["freqs"].double()
        z = torch.polar(torch.ones_like(turns), turns)[:, None, :]
        R = c["R"]

        def rotated(x, z):
            shape = x.shape[:2] + ((2, R // 2) if c["layout"] == "half" else (R // 2, 2))
            ab = x[..., :R].reshape(shape)
            ab = ab.transpose(-1, -2) if c["layout"] == "half" else ab
            r = torch.view_as_real(torch.view_as_complex(ab.contiguous()) * z)
            r = r.transpose(-1, -2) if c["layout"] == "half" else r
            return torch.cat([r.reshape(*x.shape[:2], R), x[..., R:]], -1)

        out = {}
        for name in ("q", "k"):
            if c[name] is None:
                out.update({name: None} if c["op"] == "norm_rope" else {"d" + name: None, "d" + name + "w": None})
                continue
            x, w = c[name].double(), c[name + "w"].double() + c["offset"]
            ms = x.pow(2).mean(-1, keepdim=True) + 1e-6
            if c["op"] == "norm_rope":
                out[name] = rotated(x / ms.sqrt() * w, z)
                continue
            g = rotated(c["d" + name].double(), z.conj())
            gw = g * w
            out["d" + name] = gw * ms.pow(-0.5) - x * ms.pow(-1.5) * (gw * x).mean(-1, keepdim=True)
            out["d" + name + "w"] = torch.einsum("thd,thd->d", g, x / ms.sqrt())
        return out
    if c["op"] == "cache_write":
        return {"k": _exact_quantised(c, c["k"]), "v": _exact_quantised(c, c["v"])}
    H, G = c["heads"], c["group"] if c["op"] == "attention" else 1
    if c["op"] == "cache_read":
        both = [_cached(c, b, 0, n) for b, (_, n) in enumerate(c["batch"]) if n]
        return {"k": torch.cat([k for k, _ in both]), "v": torch.cat([v for _, v in both])}
    rows, at = [], 0
    for b, (new, n) in enumerate(c["batch"]):
        if not new:
            continue
        lo = max(0, n - new + 1 - c["window"]) if c["window"] else 0
        k, v = _cached(c, b, lo, n - lo)
        q = c["q"][at:at + new].double()
        at += new
        t = torch.arange(lo, n, device=q.device)
        pos = n - new + torch.arange(new, device=q.device)[:, None]
        seen = (t <= pos) & (t > pos - (c["window"] or n + 1))
        o = torch.empty_like(q)
        for h in range(H * G):
            s = (q[:, h] * c["scale"]) @ k[:, h // G].T
            o[:, h] = torch.softmax(s.masked_fill(~seen, -math.inf), -1) @ v[:, h // G]
        rows.append(o)
    return torch.cat(rows)
