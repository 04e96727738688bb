"""Attention over the quantised cache against 64 bits, on what the cache holds.

Bounds, for a row with scores s_t, weights w_t = softmax(s)_t and A = sum w |V|
(per dimension).  K and V enter exactly.  A score is a sum over D <= 256 products: the
matrix cores' and the f32 additions' errors stay below (32 + 8) 2^-23 of
M_t = |scale| sum |q K_t|, f32 queries (two f16 parts, 11 bits each) add 2^-22 M_t,
factors and log2 e 2^-22 |s_t| <= 2^-22 M_t, the difference to the reference and the
exponential 2^-21 + 2^-22 M_t.  With delta = 64 2^-23 max M_t + 2^-20 the weights
are off by 2 delta of themselves (numerator and sum), the result by 2 delta A.
Probabilities times scale as f16: 2^-11 A for bf16 calls, 2^-22 A as two parts, and
what lies below f16's normal values at most 2^-25 of products that start at 2^6:
n 2^-31 max |V| for n positions.  Sums over tokens: (n / 32 + 100) 2^-23 A.  Then one
rounding to the type.  lse: delta + 2^-21 (|lse| + 1).

Calls that put more than 64 queries on a k / v head (of a sequence, or of the batch over a
shared prefix) take K and V times their scales as f16 values in bf16: K's rounding adds
2^-11 M_t to a score, V's and the probability's 2^-11 A each to the result.  In f16 and
f32 they take two parts of each without the product of the low ones: 2^-22 M_t and
2 2^-22 A more.
"""
import math

import pytest
import torch

import kv_reference as kr

pytestmark = pytest.mark.gpu
DT = kr.DT


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A cache of random codes and scales (its bytes outside the sequences arbitrary), the batch, the reference."""

    def __init__(self, qmv, fmt, dtype, heads, group, D, page, news, lens, seed=1, prefix=0, spread=1.0):
        self.qmv, self.fmt, self.dt, self.heads, self.group, self.D, self.page = qmv, fmt, DT[dtype], heads, group, D, page
        self.news, self.lens, self.prefix = news, lens, prefix
        B, columns = len(news), max(1, -(-max(max(lens), 1) // page))
        shared = prefix // page
        self.pages = shared + B * columns + 2
        order = torch.randperm(self.pages, generator=gen(seed))
        self.table = order[shared:shared + B * columns].view(B, columns).clone()
        self.table[:, :min(shared, columns)] = order[:min(shared, columns)]
        n = qmv.kv_cache_bytes(fmt, self.pages, heads, D, page)
        data = torch.randint(0, 256, (n,), dtype=torch.uint8, generator=gen(seed + 1))
        if fmt == "q8_0":
            data = torch.where(data == 0, torch.ones_like(data), data)
        sub = kr.set_bytes(fmt, D)
        sets = data.view(-1, sub)
        codes = D // 32 * (1024 if fmt == "q8_0" else 512)
        s = (0.5 + torch.rand((sets.shape[0], D), generator=gen(seed + 2))) / (70 if fmt == "q8_0" else 4.6)
        if spread != 1.0:
            s = s * spread ** torch.randn(s.shape, generator=gen(seed + 3))
        sets[:, codes:] = s.half().view(torch.uint8)
        self.data = data
        if prefix % page and shared < columns:  # the page in which the prefix ends: the same tokens in each
            rec = data.view(self.pages, -1)
            for b in range(1, B):
                rec[self.table[b, shared]] = rec[self.table[0, shared]]
        self.starts = [0]
        for x in news:
            self.starts.append(self.starts[-1] + x)
        self.T = self.starts[-1]
        self.q = (2 * torch.randn((max(1, self.T), heads * group, D), generator=gen(seed + 4))).to(self.dt)

    def poison(self):
        """NaN scales and arbitrary codes in every place that no sequence holds."""
        held = set()
        for b, n in enumerate(self.lens):
            for p in range(min(n, self.table.shape[1] * self.page)):
                pid = int(self.table[b, p // self.page])
                held.add((pid, p % self.page))
        half = self.data.view(torch.float16)
        for pid in range(self.pages):
            for t in range(self.page):
                if (pid, t) not in held:
                    _, _, ks, vs = kr.places(self.fmt, self.heads, self.D, self.page, pid, t)
                    half[ks] = float("nan")
                    half[vs] = -float("inf") if t % 2 else float("nan")

    def call(self, q=None, **kw):
        c = self.qmv.KVCache(self.fmt, self.pages, self.heads, self.D, self.page, data=self.data.cuda())
        q = (self.q if q is None else q).cuda()
        kw.setdefault("prefix", self.prefix)
        most = min(kw.get("max_q", -(-q.shape[0] // len(self.news))), q.shape[0])
        self.many = bool(most * self.group > 64 or (kw["prefix"] and q.shape[0] * self.group > 64))
        self.rounded = self.many and self.dt == torch.bfloat16
        return self.qmv.kv_attention(c, q, ints(self.table.tolist()), ints(self.starts), ints(self.lens), **kw)

    def sequence(self, b, n):
        """K, V [n][heads][D] in f64, and which positions are there."""
        ks, vs, there = [], [], []
        for p in range(n):
            pid = int(self.table[b, p // self.page]) if p < self.table.shape[1] * self.page else -1
            ok = 0 <= pid < self.pages
            k, v = kr.value(self.fmt, self.data, self.heads, self.D, self.page, pid if ok else 0, p % self.page)
            ks.append(k)
            vs.append(v)
            there.append(ok)
        z = torch.zeros(0, self.heads, self.D, dtype=torch.float64)
        return (torch.stack(ks) if ks else z), (torch.stack(vs) if vs else z), torch.tensor(there, dtype=torch.bool)

    def check(self, got, scale=None, window=0, lse=None, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        e, sub = kr.half_step(self.dt)
        got, worst = got.double().cpu(), 0.0
        for b, (n, ln) in enumerate(zip(self.news, self.lens)):
            if not n:
                continue
            k, v, there = self.sequence(b, max(0, ln))
            pos = torch.arange(n) + ln - n
            lo = torch.clamp(pos - window + 1, min=0) if window else torch.zeros(n, dtype=torch.long)
            for h in range(self.heads):
                r = slice(self.starts[b], self.starts[b] + n)
                g = slice(h * self.group, (h + 1) * self.group)
                kk, vv = k[:, h], v[:, h]
                keep = there.nonzero().flatten()  # absent positions are as if masked: renumber what is left
                q = self.q[r, g].double()
                t = keep
                seen = (t <= pos[:, None]) & (t >= lo[:, None]) if t.numel() else torch.zeros(n, 0, dtype=torch.bool)
                out, A, ls, M = attend(q, kk[keep], vv[keep], seen, scale)
                delta = (64 * 2.0 ** -23 + 2.0 ** -22 * self.many + 2.0 ** -11 * self.rounded) * M[..., None] + 2.0 ** -20
                count = seen.sum(-1)[:, None, None].double()
                vmax = vv[keep].abs().max() if keep.numel() else torch.zeros(())
                part = 2.0 ** -10 if self.rounded else 2.0 ** -11 if self.dt == torch.bfloat16 else 2.0 ** -22 * (1 + 2 * self.many)
                tol = A * (2 * delta + part + (count / 32 + 100) * 2.0 ** -23) + count * 2.0 ** -31 * vmax
                tol = tol + e * (out.abs() + tol) + sub
                err = (got[r, g] - out).abs()
                worst = max(worst, float((err / tol.clamp_min(1e-300)).max()))
                assert bool((err <= tol).all()), (b, h, worst)
                if lse is not None:
                    l64 = lse[r, g].double().cpu()
                    fin = torch.isfinite(ls)
                    assert torch.equal(torch.isneginf(l64), ~fin)
                    assert bool(((l64 - ls).abs()[fin] <= (delta[..., 0] + 2.0 ** -21 * (ls.abs() + 1))[fin]).all())
        say(f"  worst {worst:.3f} of the bound")


def attend(q, k, v, seen, scale):
    """(out, sum w |v|, lse, largest sum |q k| |scale|) of rows q [n][group][D] over k, v [tokens][D] (f64)."""
    s = torch.einsum("ngd,td->ngt", q * scale, k).masked_fill(~seen[:, None], -math.inf)
    m = torch.einsum("ngd,td->ngt", (q * scale).abs(), k.abs()).masked_fill(~seen[:, None], 0.0)
    if not k.shape[0]:
        z = torch.zeros(q.shape, dtype=torch.float64)
        return z, z, torch.full(q.shape[:2], -math.inf, dtype=torch.float64), z[..., 0]
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("ngt,td->ngd", w, v), torch.einsum("ngt,td->ngd", w, v.abs()), lse, m.amax(-1)


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 1000, 0, 2049]


@pytest.mark.parametrize("heads,group,D,page", [(2, 4, 64, 16), (1, 1, 32, 16), (2, 5, 96, 48), (1, 8, 128, 64), (1, 17, 64, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_single_tokens(qmv, fmt, dtype, heads, group, D, page):
    say("single", fmt, dtype, heads, group, D, page)
    c = Case(qmv, fmt, dtype, heads, group, D, page, [1 if n else 0 for n in LENS], LENS)
    for kw in (dict(), dict(max_kv=1), dict(max_kv=10 ** 9, max_q=7)):  # one part and many
        lse = torch.empty((c.T, heads * group), dtype=torch.float32, device="cuda")
        c.check(c.call(lse=lse, **kw), lse=lse)


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_every_head_size(qmv, fmt, dtype, D):
    """One and several tiles of queries, with and without a prefix (every instance of the kernel)."""
    say("head size", fmt, dtype, D)
    c = Case(qmv, fmt, dtype, 2, 3, D, 32, [1, 1, 1], [70, 200, 33], prefix=33)
    c.check(c.call())
    c.check(c.call(prefix=0))
    c = Case(qmv, fmt, dtype, 1, 2, D, 32, [23, 40], [300, 40], prefix=20)
    c.check(c.call())
    c.check(c.call(prefix=0, max_q=40, max_kv=100))


@pytest.mark.parametrize("window", [0, 1, 16, 50, 5000])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_prompt_chunks_and_windows(qmv, fmt, dtype, window):
    """Whole prompts, chunks behind a past, no tokens, more rows than tokens (rows before the first position see
    nothing)."""
    say("chunks", fmt, dtype, window)
    news, lens = [37, 1, 0, 70, 129, 20], [37, 400, 50, 333, 129, 12]
    c = Case(qmv, fmt, dtype, 2, 3, 64, 48, news, lens)
    for kw in (dict(max_q=129), dict(max_q=1, max_kv=1), dict()):
        lse = torch.empty((c.T, 6), dtype=torch.float32, device="cuda")
        got = c.call(window=window, lse=lse, **kw)
        c.check(got, window=window, lse=lse)
        assert bool((got[c.starts[5]:c.starts[5] + 8] == 0).all())


@pytest.mark.parametrize("prefix,window", [(16, 0), (100, 0), (256, 0), (100, 60), (100, 150), (700, 0), (5000, 0), (5000, 40)])
@pytest.mark.parametrize("fmt,dtype", [("q8_0", "bf16"), ("q4_0", "f16"), ("q8_0", "f32")])
def test_shared_prefix(qmv, fmt, dtype, prefix, window):
    """Sequences beyond, inside and before the prefix's end, all of it a prefix, chunks in it, windows that leave
    some or nothing of it: the same rows as without."""
    say("prefix", fmt, dtype, prefix, window)
    news, lens = [1, 1, 5, 0, 1, 40, 1], [700, 101, 120, 0, 99, 600, 1]
    c = Case(qmv, fmt, dtype, 2, 4, 64, 32, news, lens, prefix=min(prefix, 700))
    c.check(c.call(prefix=prefix, window=window), window=window)
    c.check(c.call(prefix=prefix, window=window, max_kv=1, max_q=40), window=window)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_masked_does_not_enter(qmv, fmt, dtype):
    """NaN and infinite scales and any codes behind the sequences' ends, in unused pages, and where a page id
    names none: the rows are as if they were not there."""
    news, lens = [1, 3, 30, 1], [33, 70, 45, 16]
    c = Case(qmv, fmt, dtype, 2, 4, 64, 16, news, lens)
    c.poison()
    got = c.call()
    c.check(got)
    assert bool(torch.isfinite(got).all())
    c.table[1, 2], c.table[2, 0], c.table[3, 0] = -1, c.pages, 2 ** 31 - 1  # holes, and a sequence with nothing
    got = c.call()
    c.check(got)
    assert bool((got[-1] == 0).all())
    c.check(c.call(window=20), window=20)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_what_is_masked_does_not_enter_for_many_rows(qmv, fmt, dtype):
    """The same with more rows than one block of few, over a prefix too."""
    c = Case(qmv, fmt, dtype, 2, 4, 96, 16, [1, 3, 30, 1], [33, 70, 45, 16], prefix=10)
    c.poison()
    for kw in (dict(prefix=0), dict()):
        got = c.call(max_q=30, **kw)
        c.check(got)
        assert bool(torch.isfinite(got).all())
    c.table[1, 2], c.table[2, 1] = -1, c.pages
    c.check(c.call(max_q=30, prefix=0, window=20), window=20)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [16, 17, 33, 64, 65, 128, 129])
def test_numbers_of_rows(qmv, dtype, rows):
    """About the ends of a tile, of a block and of the kernels' ranges, one part and several."""
    c = Case(qmv, "q8_0", dtype, 1, 1, 64, 32, [rows, 2], [rows + 200, 50])
    for kw in (dict(max_kv=1), dict(max_kv=rows + 200)):
        c.check(c.call(max_q=rows, **kw))
    c = Case(qmv, "q4_0", dtype, 2, 1, 32, 16, [1] * rows, [36 + i % 20 for i in range(rows)], prefix=35)
    c.check(c.call(max_q=1))


def test_table_too_short_and_numbers_out_of_order(qmv):
    c = Case(qmv, "q8_0", "bf16", 1, 2, 32, 16, [1, 1], [30, 20])
    c.lens = [100, 20]  # past the table's two columns: those positions are not there
    got = c.call()
    c.lens = [32, 20]
    c.check(got[:2])  # the position past them sees all that is
    c.lens = [2 ** 31 - 1, -2 ** 31]
    got = c.call()
    assert bool((got[1] == 0).all())
    for starts in ([0, 2, 1], [-7, 100, 2], [2, 1, 0]):
        c.starts = starts
        assert c.call().shape == c.q.shape
    torch.cuda.synchronize()


def test_special_queries_and_blocks(qmv):
    """A NaN or infinite q makes its row NaN and no other; a NaN block of V its 32 dimensions of the rows that see
    it, one of K those rows; queries of zeros and scale 0 average; far larger and smaller queries stay exact."""
    c = Case(qmv, "q8_0", "f32", 1, 2, 64, 16, [4, 1], [40, 20])
    clean = c.call()
    c.check(clean)
    bad = c.q.clone()
    bad[1, 0, 5], bad[2, 1, 63] = float("nan"), float("inf")
    got = c.call(bad)
    assert bool(torch.isnan(got[1, 0]).all()) and bool(torch.isnan(got[2, 1]).all())
    keep = torch.ones(5, 2, dtype=torch.bool)
    keep[1, 0] = keep[2, 1] = False
    assert torch.equal(got[keep], clean[keep])
    for f in (0.0, 2.0 ** -60, 2.0 ** -140):
        c.q = clean.cpu() * f
        c.check(c.call())
    c.q = torch.randn(c.q.shape, generator=gen(5)) * 1e30
    c.check(c.call(scale=1e-30), scale=1e-30)
    c.check(c.call(scale=0.0), scale=0.0)
    c.q = torch.randn(c.q.shape, generator=gen(6))
    for scale in (-0.3, 3.0):
        c.check(c.call(scale=scale), scale=scale)
    half = c.data.view(torch.float16)
    _, _, ks, vs = kr.places("q8_0", 1, 64, 16, int(c.table[0, 2]), 6)  # position 38: rows 2 and 3 see it
    was = half[vs].clone(), half[ks].clone()
    plain = c.call()
    half[vs[0, 1]] = float("nan")
    got = c.call()
    assert bool(torch.isnan(got[2:4, :, 32:]).all()) and torch.equal(got[:2], plain[:2]) and torch.equal(got[4], plain[4])
    assert bool(torch.isfinite(got[2:4, :, :32]).all())
    half[vs] = was[0]
    half[ks[0, 0]] = float("nan")
    got = c.call()
    assert bool(torch.isnan(got[2:4]).all()) and torch.equal(got[:2], plain[:2]) and torch.equal(got[4], plain[4])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_bad_blocks_of_many_rows(qmv, dtype):
    """Rows of one tile, some of which see a token whose K or V is no number: those are NaN (in the block's
    dimensions at least), the others are untouched; K and V near the ends of their range."""
    for plane in (2, 3):
        c = Case(qmv, "q8_0", dtype, 1, 3, 64, 16, [40], [75])
        clean = c.call(max_q=40)
        c.check(clean)
        half = c.data.view(torch.float16)
        at = kr.places("q8_0", 1, 64, 16, int(c.table[0, 3]), 2)[plane]  # position 50: rows 15 .. 39 see it
        half[at[0, 1]] = float("nan")
        got = c.call(max_q=40)
        assert torch.equal(got[:15], clean[:15])
        assert bool(torch.isnan(got[15:, :, 32:]).all())
    c = Case(qmv, "q4_0", dtype, 1, 3, 64, 16, [40], [75])
    sets = c.data.view(torch.float16).view(-1, kr.set_bytes("q4_0", 64) // 2)
    for scale in (60000.0, 2.0 ** -22):
        sets[:, -64:] = scale
        c.q = c.q * 0 + (2.0 ** -10 if scale > 1 else 1.0)
        sets[:, -64:-32] = scale if scale < 1 else 0.5  # K; V past what f16 holds as values
        got = c.call(max_q=40, scale=1.0)
        if dtype != "f16":  # f16 results of these sizes are infinite
            c.check(got, scale=1.0)
        else:
            assert not bool(torch.isnan(got).any())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_scales_of_any_size(qmv, dtype):
    """V's and K's scales over many powers of two, down to zero: the reference keeps products in f16's range."""
    c = Case(qmv, "q8_0", dtype, 1, 4, 64, 16, [1, 20], [500, 300], spread=8.0)
    c.data.view(-1, kr.set_bytes("q8_0", 64))[3, -64:] = 0  # scales of zero
    q = c.q
    for f in (1.0, 0.01):
        c.q = (q.float() * f).to(c.dt)
        c.check(c.call())


def test_strides_in_place_streams_and_versions(qmv):
    c = Case(qmv, "q8_0", "bf16", 2, 3, 64, 16, [1, 5, 1], [50, 20, 300])
    ref = c.call()
    wide = torch.zeros((c.T + 2, 10, 72), dtype=torch.bfloat16)
    wide[:c.T, 1:7, :64] = c.q
    dev = wide.cuda()
    cache = qmv.KVCache("q8_0", c.pages, 2, 64, 16, data=c.data.cuda())
    table, q_start, kv_len = ints(c.table.tolist()), ints(c.starts), ints(c.lens)
    q = dev[:, 1:7, :64]  # two rows behind the last sequence
    out = torch.full((6, c.T + 2, 64), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    version = out._version
    got = qmv.kv_attention(cache, q, table, q_start, kv_len, out=out, max_q=2, max_kv=304)
    assert out._version > version and bool((out[c.T:] == 7.0).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = qmv.kv_attention(cache, q[:c.T], table, q_start, kv_len, stream=side)
    side.synchronize()
    assert torch.equal(there, ref)
    c.check(got[:c.T])
    for kw in (dict(max_kv=1), dict(max_kv=304)):  # one part, and several that are joined
        keep = dev.clone()
        q = keep[:, 1:7, :64]
        want = qmv.kv_attention(cache, q, table, q_start, kv_len, max_q=2, **kw)
        assert qmv.kv_attention(cache, q, table, q_start, kv_len, out=q, max_q=2, **kw) is q
        assert torch.equal(q[:c.T], want[:c.T]) and torch.equal(q[c.T:], dev[c.T:, 1:7, :64])
        assert bool((keep[:, 0] == 0).all()) and bool((keep[:, 7:] == 0).all()) and bool((keep[:, :, 64:] == 0).all())
    with pytest.raises(ValueError, match="workspace holds"):
        qmv.kv_attention(cache, q, table, q_start, kv_len, prefix=16, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="lse must be"):
        qmv.kv_attention(cache, q, table, q_start, kv_len, lse=torch.empty(3, device="cuda"))


def test_decode_steps_as_a_graph(qmv):
    """A captured step (norms and rotary positions, cache write, attention, with and without a shared prefix) of
    growing sequences, replayed and checked against the eager step and against 64 bits each time."""
    B, hq, hk, D, page, dt = 5, 8, 2, 64, 16, torch.float32
    lens = [20, 33, 64, 47, 21]
    cache = qmv.KVCache("q8_0", B * 8, hk, D, page)
    table = torch.randperm(B * 8, generator=gen(1)).int().view(B, 8).cuda()
    table[:, 0] = table[0, 0]  # the first page is shared
    first = torch.randn((20, hk, D), generator=gen(2)).cuda()
    ints1 = lambda x: ints(x)  # noqa: E731
    for b, n in enumerate(lens):  # prompts: every sequence begins with the same tokens
        more = torch.randn((n, hk, D), generator=gen(3 + b)).cuda()
        more[:16] = first[:16]
        qmv.kv_write(cache, more, more.flip(2).contiguous(), table[b:b + 1], ints1([0, n]), ints1([n]))
    q_start, kv_len = ints1(list(range(B + 1))), ints1(lens)
    qkv = torch.randn((B, hq + 2 * hk, D), generator=gen(9)).cuda()
    qw, kw = 1 + 0.2 * torch.randn(D, generator=gen(10)).cuda(), 1 + 0.2 * torch.randn(D, generator=gen(11)).cuda()
    freqs, pos = qmv.rope_freqs(D), torch.zeros(B, dtype=torch.int64, device="cuda")

    def step(prefix, ws=None):
        q, k = qmv.norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], qw, kw, pos, freqs)
        qmv.kv_write(cache, k, qkv[:, hq + hk:], table, q_start, kv_len)
        return q, qmv.kv_attention(cache, q, table, q_start, kv_len, prefix=prefix, workspace=ws)

    graphs = []
    for prefix in (0, 16):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, prefix, step(prefix)))
    for turn in range(4):
        kv_len.add_(1)
        pos.copy_(kv_len.long() - 1)
        qkv.copy_(torch.randn(qkv.shape, generator=gen(100 + turn)))
        for g, prefix, (gq, go) in graphs:
            g.replay()
            eager = step(prefix)
            torch.cuda.synchronize()
            assert torch.equal(gq, eager[0]) and torch.equal(go, eager[1]), (turn, prefix)
            data = cache.data.cpu()
            for b in range(B):
                n = int(kv_len[b])
                kv = [kr.value("q8_0", data, hk, D, page, int(table[b, p // page]), p % page) for p in range(n)]
                for h in range(hk):
                    k, v = torch.stack([x[0][h] for x in kv]), torch.stack([x[1][h] for x in kv])
                    q = gq[b, h * 4:h * 4 + 4].double().cpu()[None]
                    out, A, _, M = attend(q, k, v, torch.ones(1, n, dtype=torch.bool), D ** -0.5)
                    tol = A * (128 * 2.0 ** -23 * M[..., None] + 2.0 ** -19 + 110 * 2.0 ** -23) + n * 2.0 ** -31 * v.abs().max()
                    assert bool(((go[b, h * 4:h * 4 + 4].double().cpu() - out[0]).abs() <= tol[0] + 2.0 ** -24 * out[0].abs()).all())


def test_repeats_and_long_cache(qmv):
    """Calls repeat bit for bit; a sequence whose pages lie past 2^32 bytes."""
    heads, D, page = 8, 128, 64
    per = qmv.kv_cache_bytes("q8_0", 1, heads, D, page)
    pages = 2 ** 32 // per + 40
    cache = qmv.KVCache("q8_0", pages, heads, D, page)
    n = 30 * page - 5
    table = torch.arange(pages - 30, pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    k, v = torch.randn((n, heads, D), generator=gen(1)), torch.randn((n, heads, D), generator=gen(2))
    qmv.kv_write(cache, k.cuda(), v.cuda(), table, ints([0, n]), ints([n]))
    q = torch.randn((1, heads * 2, D), generator=gen(3))
    a, b = (qmv.kv_attention(cache, q.cuda(), table, ints([0, 1]), ints([n])) for _ in range(2))
    assert torch.equal(a, b)
    k, v = kr.stands_for("q8_0", k), kr.stands_for("q8_0", v)
    for h in range(heads):
        out, A, _, M = attend(q[:, 2 * h:2 * h + 2].double(), k[:, h], v[:, h], torch.ones(1, n, dtype=torch.bool), D ** -0.5)
        tol = A * (128 * 2.0 ** -23 * M[..., None] + 2.0 ** -19 + (n / 32 + 100) * 2.0 ** -23) + n * 2.0 ** -31 * v[:, h].abs().max()
        assert bool(((a[:, 2 * h:2 * h + 2].double().cpu() - out).abs() <= tol + 2.0 ** -24 * out.abs()).all())


@pytest.mark.parametrize("prefix,max_kv", [(0, 1), (0, 700), (16, 700)])
def test_rows_before_the_first_sequence(qmv, prefix, max_kv):
    """A call on some sequences of a larger batch: q_start begins past 0; with one part and with a join."""
    c = Case(qmv, "q8_0", "f32", 2, 3, 64, 16, [2, 1, 3], [700, 20, 40], prefix=prefix)
    cache = qmv.KVCache("q8_0", c.pages, 2, 64, 16, data=c.data.cuda())
    table, kv_len, q = ints(c.table.tolist()), ints(c.lens), torch.cat([c.q.new_full((5, 6, 64), 9.0), c.q, c.q[:2]]).cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((13, 6), 7.0, device="cuda")
    qmv.kv_attention(cache, q, table, ints([s + 5 for s in c.starts]), kv_len, prefix=prefix, max_q=3, max_kv=max_kv, out=out, lse=lse)
    for x in (out, lse):
        assert bool((x[:5] == 7.0).all()) and bool((x[11:] == 7.0).all())
    c.many, c.rounded = bool(prefix), False
    c.check(out[5:11], lse=lse[5:11])
    kk, vv = torch.full((13, 2, 64), 7.0, device="cuda"), torch.full((13, 2, 64), 7.0, device="cuda")
    before = c.data.clone()
    qmv.kv_read(cache, table, ints([s + 5 for s in c.starts]), kv_len, 13, k=kk, v=vv)
    assert bool((kk[:5] == 7.0).all()) and bool((vv[11:] == 7.0).all())
    qmv.kv_write(cache, kk, vv, table, ints([s + 5 for s in c.starts]), kv_len)
    again = qmv.kv_read(cache, table, ints([s + 5 for s in c.starts]), kv_len, 13, dtype=torch.float32)
    assert bool(((again[0][5:11] - kk[5:11]).abs() <= kk[5:11].abs().amax() / 100).all())  # quantised twice: a step at most
    held = cache.data.cpu()
    assert int((held != before).sum()) <= 6 * 2 * 2 * (64 + 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_negative_scales(qmv, fmt, dtype):
    """Blocks that another program wrote: scales of either sign, the largest of them positive and next to f16's end
    (products past f16's range if the exponent were taken from the negative ones), few rows and many."""
    for news in ([1, 2], [1, 40]):
        c = Case(qmv, fmt, dtype, 2, 2, 64, 16, news, [70, 300], seed=3)
        sub, codes = kr.set_bytes(fmt, 64), 2 * (1024 if fmt == "q8_0" else 512)
        half = c.data.view(-1, sub)[:, codes:].view(torch.float16)
        v = half[:, half.shape[1] // 2:]
        sign = torch.where(torch.rand(half.shape, generator=gen(5)) < 0.5, -1.0, 1.0)
        size = torch.where(sign > 0, 500.0, 1 / 1024)[:, half.shape[1] // 2:]
        v.copy_((v.float() * size).half())
        half.copy_((half.float() * sign).half())
        c.check(c.call(max_q=max(news), max_kv=300))


@pytest.mark.parametrize("group", [2, 33])
def test_prefix_of_a_batch_with_many_sequences_without_rows(qmv, group):
    """Rows whose sequences lie far apart, next to each other and last, in the kernels for few and for many rows."""
    news, lens = [0] * 300, [20 + b % 7 for b in range(300)]
    for b in (0, 90, 91, 200, 299):
        news[b] = 1
    news[91] = 2
    c = Case(qmv, "q8_0", "f32", 1, group, 32, 16, news, lens, prefix=16)
    c.check(c.call(max_q=2))


def test_first_call_of_a_process_in_a_capture():
    """Nothing that a first call sets up gets in the way of a capture."""
    import os
    import subprocess
    import sys
    code = """
import torch, gemm_dequant_matvec_amd as qmv
dev = "cuda"
q = torch.randn(3000, 4, 64, device=dev).half(); k = torch.randn(3000, 2, 64, device=dev).half()
pos, f = torch.arange(3000, device=dev), qmv.rope_freqs(64)
c = qmv.KVCache("q8_0", 40, 2, 64, 128)
c.data.zero_()
t = torch.arange(40, device=dev).int()[None].contiguous()
n = torch.tensor([3000], dtype=torch.int32, device=dev)
s = torch.tensor([0, 3000], dtype=torch.int32, device=dev)
torch.cuda.synchronize()
def step():
    a, b = qmv.norm_rope(q, k, None, None, pos, f)
    qmv.kv_write(c, b, k, t, s, n)
    return qmv.kv_attention(c, a, t, s, n), qmv.norm_rope_backward(q, k, None, None, a, b, pos, f)[0]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
for turn in range(3):
    q.normal_(); k.normal_()
    g.replay()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, want)), turn
print("captured first")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=90, cwd=root)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
