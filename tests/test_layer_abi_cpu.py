"""The many-token layer operators without a GPU: exports, every refusal (found
on the host, before any launch), workspace sizes, and the rotary frequencies."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qmv_layer.h")
OK, NULL, FORMAT, UNSUP, SHAPE, ALIGN, DTYPE, OVER = 0, -1, -2, -3, -4, -5, -6, -7


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


def test_exports(q):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(qmv_[a-z0-9_]+)\s*\(", text))
    lib = ctypes.CDLL(q.LIB_PATH)
    assert names == set(q.LAYER_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


P = 0x10000  # an aligned address that no refused call touches


def glu(q, **kw):
    a = dict(fmt=2, N=64, K=64, M=4, wg=P, wu=P, x=P, xd=3, act=1, h=3 * P, hd=3, g=0, u=0)
    a.update(kw)
    return q.raw_call("qmv_gemm_glu", a["fmt"], a["N"], a["K"], a["M"], a["wg"], a["wu"], a["x"], a["xd"], a["act"],
                      a["h"], a["hd"], a["g"], a["u"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(fmt=10), FORMAT, "10"), (dict(N=0), SHAPE, "N=0"), (dict(K=0), SHAPE, "K=0"), (dict(K=96), SHAPE, "K=96"),
    (dict(M=0), SHAPE, "M=0"), (dict(wg=0), NULL, "W_gate"), (dict(wu=0), NULL, "W_up"), (dict(x=0), NULL, "X"),
    (dict(h=0), NULL, "H"), (dict(g=P), NULL, "U"), (dict(u=P), NULL, "G"), (dict(xd=9), DTYPE, "x_dtype"),
    (dict(hd=9), DTYPE, "h_dtype"), (dict(xd=1), UNSUP, "bf16"), (dict(xd=4), UNSUP, "bf16"), (dict(hd=2), UNSUP, "h_dtype"),
    (dict(act=0), UNSUP, "act"), (dict(act=4), UNSUP, "act"), (dict(wg=P + 4), ALIGN, "W_gate"),
    (dict(wu=P + 8), ALIGN, "W_up"), (dict(x=P + 2), ALIGN, "X"), (dict(h=P + 8), ALIGN, "H"),
    (dict(g=P + 2, u=P), ALIGN, "G"), (dict(g=P, u=P + 2), ALIGN, "U"), (dict(M=1 << 33), OVER, "M"),
    (dict(N=1 << 31), OVER, "N"), (dict(M=1 << 24, N=1 << 20), OVER, "M * N"),
    (dict(M=(1 << 30) + 1, N=1), OVER, "M is past"), (dict(N=1 << 22), OVER, "2^21")])
def test_glu_refusals(q, kw, status, text):
    assert glu(q, **kw) == status, q.last_error()
    assert text in q.last_error()


@pytest.mark.parametrize("kw,text", [(dict(h=P), "X"), (dict(g=P, u=4 * P), "X"), (dict(g=3 * P, u=4 * P), "one buffer"),
                                     (dict(g=4 * P, u=4 * P), "one buffer")])
def test_glu_buffers_given_twice(q, kw, text):
    assert glu(q, **{"h": 3 * P, **kw}) == UNSUP and text in q.last_error()


def bwd(q, **kw):
    a = dict(fmt=2, N=64, K=64, M=4, wg=P, wu=P, g=P, u=2 * P, dh=3 * P, d=3, act=1, dg=4 * P, du=5 * P, dx=6 * P, ws=0,
             nb=0)
    a.update(kw)
    return q.raw_call("qmv_gemm_glu_backward", a["fmt"], a["N"], a["K"], a["M"], a["wg"], a["wu"], a["g"], a["u"],
                      a["dh"], a["d"], a["act"], a["dg"], a["du"], a["dx"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(fmt=0), FORMAT, "0"), (dict(K=32), SHAPE, "K=32"), (dict(M=-1), SHAPE, "M=-1"), (dict(wg=0), NULL, "W_gate"),
    (dict(g=0), NULL, "G"), (dict(u=0), NULL, "U"), (dict(dh=0), NULL, "dH"), (dict(dg=0), NULL, "dG"),
    (dict(du=0), NULL, "dU"), (dict(dx=0), NULL, "dX"), (dict(d=1), UNSUP, "bf16"), (dict(d=0), DTYPE, "dtype"),
    (dict(act=7), UNSUP, "act"), (dict(g=P + 2), ALIGN, "G"), (dict(dx=6 * P + 8), ALIGN, "dX"),
    (dict(du=4 * P), UNSUP, "dG and dU"), (dict(dx=P), UNSUP, "dX is the buffer of G"),
    (dict(dx=4 * P), UNSUP, "dX is the buffer of dG")])
def test_backward_refusals(q, kw, status, text):
    assert bwd(q, **kw) == status, q.last_error()
    assert text in q.last_error()


def test_backward_workspace(q):
    """A shape with split sums refuses a missing, short or misaligned workspace."""
    big = dict(N=5632, K=2048, M=4)
    need = q.gemm_glu_backward_bytes("w4a16_g64", 5632, 2048, 4)
    assert need > 0 and need % (4 * 2048 * 4) == 0
    assert bwd(q, **big) == NULL and "ws" in q.last_error()
    assert bwd(q, **big, ws=7 * P, nb=need - 1) == SHAPE and str(need) in q.last_error()
    assert bwd(q, **big, ws=7 * P + 8, nb=need) == ALIGN
    out = ctypes.c_size_t()
    assert q.raw_call("qmv_gemm_glu_backward_bytes", 2, 64, 64, 4, None) == NULL
    assert q.raw_call("qmv_gemm_glu_backward_bytes", 2, 64, 65, 4, ctypes.byref(out)) == SHAPE
    assert q.raw_call("qmv_gemm_glu_backward_bytes", 2, 64, 1 << 30, 1 << 30, ctypes.byref(out)) == OVER
    # many tiles of their own: no split, no workspace
    assert q.gemm_glu_backward_bytes("w4a16_g64", 5632, 4096, 65536) == 0


def rope(q, tensors=None, **kw):
    a = dict(T=4, D=64, R=64, layout=1, dtype=3, pos=P, freqs=P)
    a.update(kw)
    ts = [dict()] if tensors is None else tensors
    arr = (q.QmvRopeTensor * max(1, len(ts)))()
    for i, t in enumerate(ts):
        v = dict(x=P, y=2 * P, heads=2, x_token=128, x_head=64, y_token=128, y_head=64)
        v.update(t)
        for n, x in v.items():
            setattr(arr[i], n, x)
    return q.raw_call("qmv_rope", a["T"], a["D"], a["R"], a["layout"], a.get("count", len(ts)),
                      None if a.get("no_tensors") else arr, a["dtype"], a["pos"], a["freqs"], 1.0, 0, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(T=0), SHAPE, "T=0"), (dict(D=0), SHAPE, "D=0"), (dict(R=0), SHAPE, "R=0"), (dict(R=3), SHAPE, "R=3"),
    (dict(R=66), SHAPE, "R=66"), (dict(D=8192, R=4098), SHAPE, "R=4098"), (dict(layout=0), UNSUP, "layout"),
    (dict(layout=3), UNSUP, "layout"), (dict(count=0), SHAPE, "count"), (dict(count=5), SHAPE, "count"),
    (dict(no_tensors=True), NULL, "tensors"), (dict(pos=0), NULL, "pos"), (dict(freqs=0), NULL, "freqs"),
    (dict(dtype=0), DTYPE, "dtype"), (dict(dtype=4), UNSUP, "rope"), (dict(pos=P + 4), ALIGN, "pos"),
    (dict(freqs=P + 2), ALIGN, "freqs"), (dict(T=1 << 31), OVER, "T"),
    (dict(tensors=[dict(x=0)]), NULL, "tensors[0].x"), (dict(tensors=[{}, dict(y=0)]), NULL, "tensors[1].y"),
    (dict(tensors=[dict(heads=0)]), SHAPE, "heads=0"), (dict(tensors=[dict(x=P + 1)]), ALIGN, "tensors[0].x"),
    (dict(dtype=1, tensors=[dict(y=P + 2)]), ALIGN, "tensors[0].y"),
    (dict(tensors=[dict(y=P, y_token=256)]), UNSUP, "in place"), (dict(tensors=[dict(heads=1 << 31)]), OVER, "heads"),
    (dict(D=1 << 20, tensors=[dict(heads=1 << 12)]), OVER, "heads")])
def test_rope_refusals(q, kw, status, text):
    assert rope(q, **kw) == status, q.last_error()
    assert text in q.last_error()


def test_binding_checks(q):
    """Shapes, types and sizes that the pointers alone would not show."""
    W1 = torch.zeros(q.packed_bytes("w4a16_g64", 64, 128), dtype=torch.uint8)
    X = torch.zeros(4, 128, dtype=torch.bfloat16)
    g = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad in (lambda: q.gemm_glu("w4a16_g64", W1, W1[:-256], X, 64, 128),
                lambda: q.gemm_glu("w4a16_g64", W1, W1, X[:, :64], 64, 128),
                lambda: q.gemm_glu("w4a16_g64", W1, W1, X, 64, 128, act="tanh"),
                lambda: q.gemm_glu("w4a16_g64", W1, W1, X, 64, 128, G=g),
                lambda: q.gemm_glu("w4a16_g64", W1, W1, X, 64, 128, H=g.half()),
                lambda: q.gemm_glu("w4a16_g64", W1, W1, X, 64, 128, H=g[:3]),
                lambda: q.gemm_glu("w4a16_g64", W1, W1, X, 64, 128),  # not on the GPU
                lambda: q.gemm_glu_backward("w4a16_g64", W1, W1, g, g[:3], g, 64, 128),
                lambda: q.gemm_glu_backward("w4a16_g64", W1, W1, g, g, g.half(), 64, 128),
                lambda: q.gemm_glu_backward("w4a16_g64", W1, W1, g, g, g, 64, 128, dX=g),
                lambda: q.rope(X, None, torch.zeros(4, dtype=torch.int64), torch.zeros(8)),
                lambda: q.rope(X.view(4, 2, 64), X.view(4, 4, 32), torch.zeros(4, dtype=torch.int64), torch.zeros(8)),
                lambda: q.rope(X.view(4, 2, 64), None, torch.zeros(4), torch.zeros(8)),
                lambda: q.rope(X.view(4, 2, 64), None, torch.zeros(3, dtype=torch.int64), torch.zeros(8)),
                lambda: q.rope(X.view(4, 2, 64), None, torch.zeros(4, dtype=torch.int64), torch.zeros(8), layout="neox"),
                lambda: q.rope(X.view(4, 2, 64), None, torch.zeros(4, dtype=torch.int64), torch.zeros(8))):
        with pytest.raises(ValueError):
            bad()


def test_rope_freqs(q):
    R, base = 64, 10000.0
    i = np.arange(R // 2)
    f = base ** (-2.0 * i / R)
    get = lambda **kw: q.rope_freqs(R, base, device="cpu", **kw).numpy()  # noqa: E731
    assert np.array_equal(get(), f.astype(np.float32))
    assert np.array_equal(get(scaling="linear", factor=4.0), (f / 4).astype(np.float32))
    ntk = (base * 8.0 ** (R / (R - 2))) ** (-2.0 * i / R)
    np.testing.assert_allclose(get(scaling="ntk", factor=8.0), ntk, rtol=2.0 ** -23)
    # the slowest pair of the stretched base turns 8 times slower
    np.testing.assert_allclose(get(scaling="ntk", factor=8.0)[-1], f[-1] / 8, rtol=2.0 ** -22)
    p = get(scaling="parts", factor=4.0, original=2048.0, low=1.0, high=32.0)
    turns = 2048.0 * f / (2 * math.pi)
    assert np.array_equal(p[turns >= 32], f.astype(np.float32)[turns >= 32]) and (turns >= 32).any()
    assert np.array_equal(p[turns <= 1], (f / 4).astype(np.float32)[turns <= 1]) and (turns <= 1).any()
    mid = (turns > 1) & (turns < 32)
    c = (turns - 1) / 31
    np.testing.assert_allclose(p[mid], (f * (c + (1 - c) / 4))[mid], rtol=2.0 ** -23)


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), SHAPE), (dict(R=7), SHAPE), (dict(R=4098), SHAPE), (dict(R=2, scaling="ntk", factor=2.0), SHAPE),
    (dict(R=8, base=0.0), UNSUP), (dict(R=8, base=float("nan")), UNSUP), (dict(R=8, scaling="linear", factor=0.5), UNSUP),
    (dict(R=8, scaling="parts", factor=2.0), UNSUP),
    (dict(R=8, scaling="parts", factor=2.0, original=64.0, low=4.0, high=4.0), UNSUP)])
def test_rope_freqs_refusals(q, kw, status):
    with pytest.raises(q.QmvError) as e:
        q.rope_freqs(device="cpu", **kw)
    assert e.value.status == status


def test_rope_freqs_unknown_kind(q):
    with pytest.raises(ValueError):
        q.rope_freqs(8, scaling="dynamic", device="cpu")
    sc = q.QmvRopeScaling(9, 2.0, 0.0, 0.0, 0.0)
    out = (ctypes.c_float * 4)()
    assert q.raw_call("qmv_rope_freqs", 8, ctypes.c_double(1e4), ctypes.byref(sc), out) == UNSUP
    assert q.raw_call("qmv_rope_freqs", 8, ctypes.c_double(1e4), None, None) == NULL
