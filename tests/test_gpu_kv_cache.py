"""Writing and reading the quantised cache, bit for bit: the steps of the
quantisation are single f32 operations, and what a code stands for is exact."""
import pytest
import torch

import kv_reference as kr

pytestmark = pytest.mark.gpu
DT = kr.DT


def say(*a):
    print(*a, flush=True)


def randn(shape, dt, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dt)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def batch(news, lens):
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    return ints(starts), ints(lens)


def filled(qmv, fmt, pages, heads, D, page, seed):
    """A cache of arbitrary bytes."""
    c = qmv.KVCache(fmt, pages, heads, D, page)
    c.data.copy_(torch.randint(0, 256, (c.data.numel(),), dtype=torch.uint8, generator=torch.Generator().manual_seed(seed)))
    return c


def expected(fmt, before, heads, D, page, table, news, lens, k, v, pages):
    """The bytes after writing, token by token."""
    data = before.clone()
    half = data.view(torch.float16)
    row = 0
    for b, (n, ln) in enumerate(zip(news, lens)):
        for i in range(n):
            p = ln - n + i
            if 0 <= p < len(table[b]) * page and 0 <= table[b][p // page] < pages:
                ki, vi, ks, vs = kr.places(fmt, heads, D, page, table[b][p // page], p % page)
                e = torch.arange(D) % 32
                for x, ci, si, high in ((k[row], ki, ks, e % 8 >= 4), (v[row], vi, vs, e >= 16)):
                    q, d = kr.quantised(fmt, x)
                    if fmt == "q8_0":
                        data[ci] = (q + 128).to(torch.uint8)
                    else:
                        q = (q + 8).to(torch.uint8)
                        data[ci[:, ~high]] = q[:, ~high] | (q[:, high] << 4)
                    half[si] = d
            row += 1
    return data


def same_bytes(got, want, fmt):
    got = got.cpu()
    bad = (got != want).nonzero().flatten()
    say(f"  {fmt}: {bad.numel()} of {want.numel()} bytes differ")
    assert bad.numel() == 0, bad[:8].tolist()


# (new tokens, lengths with them): single tokens at every place of a group and a set, prompts that begin
# and end within groups, sets and pages, no tokens, one sequence
NEWS = {"one": ([1], [1]), "steps": ([1] * 9, [1, 2, 3, 4, 5, 16, 17, 64, 65]), "prompts": ([5, 0, 33, 1, 130], [5, 7, 40, 90, 131]),
        "long": ([300], [303])}


@pytest.mark.parametrize("heads,D,page", [(1, 32, 16), (3, 96, 48), (4, 64, 16), (2, 128, 64), (1, 256, 32), (2, 160, 112)])
@pytest.mark.parametrize("case", sorted(NEWS))
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_bytes_and_values(qmv, fmt, dtype, case, heads, D, page):
    news, lens = NEWS[case]
    say("kv_write", fmt, dtype, case, heads, D, page)
    columns = max(1, -(-max(lens) // page))
    pages = len(news) * columns + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:len(news) * columns]
    table = order.view(len(news), columns).tolist()
    T = sum(news)
    k, v = randn((T, heads, D), DT[dtype], 2, 3.0), randn((T, heads, D), DT[dtype], 3)
    c = filled(qmv, fmt, pages, heads, D, page, 4)
    before = c.data.cpu()
    q_start, kv_len = batch(news, lens)
    qmv.kv_write(c, k.cuda(), v.cuda(), ints(table), q_start, kv_len)
    same_bytes(c.data, expected(fmt, before, heads, D, page, table, news, lens, k, v, pages), fmt)
    for out in ("f32", "bf16", "f16"):
        got = qmv.kv_read(c, ints(table), q_start, kv_len, T, dtype=DT[out])
        for g, x in zip(got, (k, v)):
            assert torch.equal(g.cpu(), kr.stands_for(fmt, x).to(DT[out])), out


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_special_blocks(qmv, fmt):
    """Zeros, ties, the largest and smallest values, scales past f16 and below it, NaN and infinities: the
    definition's bits, and neighbours of a bad block are whole."""
    D, rows = 64, 12
    x = randn((rows, 1, D), torch.float32, 5)
    x[0] = 0
    x[1, 0, :32] = torch.arange(32) - 15.5  # ties at d = 15.5 / 127 are none, at d = 1 below
    x[2, 0, :32] = (torch.arange(32) % 16 - 7.5)
    x[2, 0, 0] = 127.0 if fmt == "q8_0" else 7.5  # d = 1: halves round to even
    x[3] *= 3e38 / x[3].abs().max()
    x[4] *= 1e-6 / x[4].abs().max()  # scales are f16 subnormals
    x[5] *= 1e-12
    x[6] = -x[6].abs().max()
    x[7, 0, 3] = float("nan")
    x[8, 0, 40] = float("inf")
    x[9, 0, 40] = -float("inf")
    x[10] = 2.0 ** -149
    x[11, 0, 0] = 65504.0 * (127 if fmt == "q8_0" else 7.5) * 1.01
    c = filled(qmv, fmt, 1, 1, D, 16, 6)
    table, (q_start, kv_len) = ints([[0]]), batch([rows], [rows])
    qmv.kv_write(c, x.cuda(), x.flip(0).contiguous().cuda(), table, q_start, kv_len)
    k, v = qmv.kv_read(c, table, q_start, kv_len, rows, dtype=torch.float32)
    for got, want in ((k.cpu(), kr.stands_for(fmt, x)), (v.cpu(), kr.stands_for(fmt, x.flip(0)))):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.double(), nan=0.0), torch.nan_to_num(want, nan=0.0).float().double())
    assert bool(torch.isnan(k[7, 0, :32]).all()) and not bool(torch.isnan(k[7, 0, 32:]).any())


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_absent_places_and_rows(qmv, fmt):
    """Page ids that are none, positions past the table and below 0, rows behind the last sequence: nothing is
    written there or read from there, rows of a sequence give zeros and others stay."""
    heads, D, page, pages = 2, 32, 16, 6
    table = [[3, -1], [pages, 4], [0, 1], [2 ** 31 - 1, -2 ** 31]]
    news, lens = [20, 18, 10, 3], [20, 19, 40, 2]
    T = sum(news) + 5
    k, v = randn((T, heads, D), torch.bfloat16, 7), randn((T, heads, D), torch.bfloat16, 8)
    c = filled(qmv, fmt, pages, heads, D, page, 9)
    before = c.data.cpu()
    q_start, kv_len = batch(news, lens)
    qmv.kv_write(c, k.cuda(), v.cuda(), ints(table), q_start, kv_len)
    same_bytes(c.data, expected(fmt, before, heads, D, page, table, news, lens, k, v, pages), fmt)
    out = torch.full((2, T, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qmv.kv_read(c, ints(table), q_start, kv_len, T, k=out[0], v=out[1])
    row = 0
    for b, (n, ln) in enumerate(zip(news, lens)):
        for i in range(n):
            p = ln - n + i
            there = 0 <= p < 2 * page and 0 <= table[b][p // page] < pages
            want = kr.stands_for(fmt, torch.stack([k[row], v[row]])).bfloat16() if there else torch.zeros(2, heads, D)
            assert torch.equal(out[:, row].cpu().float(), want.float()), (b, i, there)
            row += 1
    assert bool((out[:, sum(news):] == 7.0).all())


def test_numbers_out_of_order_stay_in_bounds(qmv):
    """A q_start that falls, or names rows that are not there, reaches no row outside the call's."""
    c = filled(qmv, "q8_0", 4, 1, 32, 16, 10)
    k = randn((8, 1, 32), torch.float32, 11).cuda()
    for starts in ([0, 6, 3, 8], [-5, 2, 100, 7], [9, 9, 9, 9], [2 ** 31 - 1, -2 ** 31, 5, 4]):
        qmv.kv_write(c, k, k, ints([[0, 1], [2, 3], [1, 2]]), ints(starts), ints([20, 2 ** 31 - 1, -2 ** 31]))
        out = qmv.kv_read(c, ints([[0, 1], [2, 3], [1, 2]]), ints(starts), ints([20, 2 ** 31 - 1, -2 ** 31]), 8)
        torch.cuda.synchronize()
        assert out[0].shape == (8, 1, 32)


def test_strides_streams_and_graph(qmv):
    """k and v out of one fused product and head-major, into strided outputs, on another stream, and a captured
    write and read that follow the lengths on the device."""
    heads, D, page, B = 3, 64, 16, 4
    fused = randn((B, 2 * heads + 1, D), torch.float16, 12).cuda()
    k, v = fused[:, 1:heads + 1], fused[:, heads + 1:]
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    q_start, kv_len = batch([1] * B, [1, 17, 33, 60])
    a, b = (filled(qmv, "q4_0", B * 4, heads, D, page, 13) for _ in range(2))
    qmv.kv_write(a, k, v, table, q_start, kv_len)
    hm = k.transpose(0, 1).contiguous().transpose(0, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmv.kv_write(b, hm, v, table, q_start, kv_len, stream=side)
    side.synchronize()
    assert torch.equal(a.data, b.data)
    wide = torch.full((B, 2 * heads, D + 8), 7.0, dtype=torch.float16, device="cuda")
    qmv.kv_read(a, table, q_start, kv_len, B, k=wide[:, :heads, :D], v=wide[:, heads:, :D])
    plain = qmv.kv_read(a, table, q_start, kv_len, B, dtype=torch.float16)
    assert torch.equal(wide[:, :heads, :D], plain[0]) and torch.equal(wide[:, heads:, :D], plain[1])
    assert bool((wide[:, :, D:] == 7.0).all())
    big = torch.cat([table, table], 1)[:, :4]  # rows of a wider table
    c = filled(qmv, "q4_0", B * 4, heads, D, page, 13)
    qmv.kv_write(c, k, v, big, q_start, kv_len)
    assert torch.equal(a.data, c.data)
    g, kk, vv = torch.cuda.CUDAGraph(), k.clone(), v.clone()
    version = a.data._version
    with torch.cuda.graph(g):
        qmv.kv_write(a, kk, vv, table, q_start, kv_len)
        out = qmv.kv_read(a, table, q_start, kv_len, B, dtype=torch.float32)
    assert a.data._version > version
    for turn in range(4):
        kv_len.add_(1)
        kk.mul_(1.5)
        g.replay()
        qmv.kv_write(c, kk, vv, table, q_start, kv_len)
        eager = qmv.kv_read(c, table, q_start, kv_len, B, dtype=torch.float32)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, eager)), turn


@pytest.mark.parametrize("B", [64, 65, 300, 5000])
def test_many_sequences(qmv, B):
    """The search for a row's sequence over one, two and three steps of 64."""
    g = torch.Generator().manual_seed(B)
    news = torch.randint(0, 4, (B,), generator=g).tolist()
    lens = [n + int(e) for n, e in zip(news, torch.randint(0, 13, (B,), generator=g))]
    T = sum(news)
    k, v = randn((T, 1, 32), torch.float32, 14).cuda(), randn((T, 1, 32), torch.float32, 15).cuda()
    c = filled(qmv, "q8_0", B, 1, 32, 16, 16)
    table, (q_start, kv_len) = ints([[b] for b in range(B)]), batch(news, lens)
    qmv.kv_write(c, k, v, table, q_start, kv_len)
    kk, vv = qmv.kv_read(c, table, q_start, kv_len, T, dtype=torch.float32)
    assert torch.equal(kk.cpu().double(), kr.stands_for("q8_0", k.cpu())) and torch.equal(vv.cpu().double(), kr.stands_for("q8_0", v.cpu()))


def test_more_sets_than_workgroups(qmv):
    """More sequences than one launch has workgroups for: each takes several sets."""
    B = 530000
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((B, 1, 32), device="cuda", generator=g) for _ in range(2))
    c = qmv.KVCache("q4_0", B, 1, 32, 16)
    c.data.zero_()
    table = torch.randperm(B, device="cuda", generator=g).int()[:, None].contiguous()
    q_start, kv_len = torch.arange(B + 1, device="cuda").int(), (torch.arange(B, device="cuda") % 16 + 1).int()
    qmv.kv_write(c, k, v, table, q_start, kv_len)
    kk, vv = qmv.kv_read(c, table, q_start, kv_len, B, dtype=torch.float32)
    for got, x in ((kk, k), (vv, v)):
        assert torch.equal(got.cpu().double(), kr.stands_for("q4_0", x.cpu()))


def test_past_2_32_bytes(qmv):
    """Pages whose bytes lie past 32-bit offsets."""
    heads, D, page = 8, 128, 64
    per = qmv.kv_cache_bytes("q8_0", 1, heads, D, page)
    pages = 2 ** 32 // per + 100
    say("cache of", pages, "pages,", pages * per, "bytes")
    c = qmv.KVCache("q8_0", pages, heads, D, page)
    table, (q_start, kv_len) = ints([[pages - 1, pages - 60]]), batch([100], [100])
    k, v = randn((100, heads, D), torch.float32, 17), randn((100, heads, D), torch.float32, 18)
    qmv.kv_write(c, k.cuda(), v.cuda(), table, q_start, kv_len)
    kk, vv = qmv.kv_read(c, table, q_start, kv_len, 100, dtype=torch.float32)
    assert torch.equal(kk.cpu().double(), kr.stands_for("q8_0", k)) and torch.equal(vv.cpu().double(), kr.stands_for("q8_0", v))
    tail = c.data.view(pages, -1)[pages - 1].cpu()
    assert torch.equal(kr.value("q8_0", tail, heads, D, page, 0, 5)[0], kr.stands_for("q8_0", k[5]))
