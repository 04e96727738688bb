"""The normed heads with rotary positions without a GPU: every refusal is found on
the host, before any launch; workspace sizes."""
import ctypes
import struct

import pytest
import torch

OK, NULL, UNSUP, SHAPE, ALIGN, DTYPE, OVER = 0, -1, -3, -4, -5, -6, -7
P = 0x100000  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


T1 = dict(x=P, y=2 * P, w=3 * P, heads=2, xt=128, xh=64, yt=128, yh=64)
G1 = dict(x=P, dy=2 * P, dx=3 * P, w=4 * P, dw=5 * P, heads=2, xt=128, xh=64, gt=128, gh=64, yt=128, yh=64)


def fwd(q, tensors=None, **kw):
    a = dict(T=4, D=64, R=64, layout=1, count=None, dtype=3, wd=3, eps=1e-6, off=0.0, pos=P, freqs=P, tens=True)
    a.update(kw)
    ts = [dict(T1, **t) for t in (tensors or [{}])]
    raw = b"".join(struct.pack("8q", *t.values()) for t in ts)
    return q.raw_call("qmv_norm_rope", a["T"], a["D"], a["R"], a["layout"], a["count"] or len(ts), raw if a["tens"] else None,
                      a["dtype"], a["wd"], a["eps"], a["off"], a["pos"], a["freqs"], 1.0, None)


def bwd(q, tensors=None, **kw):
    a = dict(T=4, D=64, R=64, layout=1, dtype=3, wd=3, eps=1e-6, off=0.0, pos=P, freqs=P, ws=16 * P, nb=1 << 20)
    a.update(kw)
    ts = [dict(G1, **t) for t in (tensors or [{}])]
    raw = b"".join(struct.pack("12q", *t.values()) for t in ts)
    return q.raw_call("qmv_norm_rope_backward", a["T"], a["D"], a["R"], a["layout"], len(ts), raw, a["dtype"], a["wd"],
                      a["eps"], a["off"], a["pos"], a["freqs"], 1.0, a["ws"], a["nb"], None)


COMMON = [(dict(T=0), SHAPE, "T=0"), (dict(D=0), SHAPE, "D=0"), (dict(D=1025), SHAPE, "1025"), (dict(R=0), SHAPE, "R=0"),
          (dict(R=3), SHAPE, "R=3"), (dict(R=66), SHAPE, "R=66"), (dict(layout=3), UNSUP, "layout"),
          (dict(dtype=9), DTYPE, "dtype"), (dict(dtype=4, wd=4), UNSUP, "f32"), (dict(wd=2), DTYPE, "w_dtype"),
          (dict(eps=-1.0), UNSUP, "eps"), (dict(eps=float("nan")), UNSUP, "eps"), (dict(off=float("inf")), UNSUP, "w_offset"),
          (dict(pos=0), NULL, "pos"), (dict(freqs=0), NULL, "freqs"), (dict(pos=P + 4), ALIGN, "pos"),
          (dict(freqs=P + 2), ALIGN, "freqs"), (dict(T=1 << 31), OVER, "T"),
          (dict(tensors=[dict(heads=0)]), SHAPE, "heads"), (dict(tensors=[dict(heads=1 << 29)]), OVER, "heads"),
          (dict(tensors=[dict(heads=1 << 27)]), OVER, "heads"),
          (dict(tensors=[dict(x=0)]), NULL, "x"), (dict(tensors=[dict(x=P + 1)]), ALIGN, "x"),
          (dict(tensors=[dict(w=P + 1)]), ALIGN, "weight"), (dict(wd=1, tensors=[dict(w=3 * P + 2)]), ALIGN, "weight"),
          (dict(tensors=[dict(yt=64)]), UNSUP, "more than once"), (dict(tensors=[dict(yh=32)]), UNSUP, "more than once")]


@pytest.mark.parametrize("kw,status,text", COMMON + [
    (dict(tens=False), NULL, "tensors"), (dict(count=5), SHAPE, "count"), (dict(count=-1), SHAPE, "count"),
    (dict(tensors=[dict(y=0)]), NULL, "y"), (dict(tensors=[dict(y=P + 1)]), ALIGN, "y"),
    (dict(tensors=[dict(y=P, yt=256)]), UNSUP, "in place"), (dict(tensors=[dict(y=3 * P)]), UNSUP, "weight"),
    (dict(tensors=[{}, dict(x=5 * P)]), UNSUP, "one buffer"),
    (dict(tensors=[{}, dict(x=5 * P, y=P)]), UNSUP, "tensors[0].x")])
def test_forward_refusals(q, kw, status, text):
    assert fwd(q, **kw) == status, q.last_error()
    assert text in q.last_error()


@pytest.mark.parametrize("kw,status,text", COMMON + [
    (dict(tensors=[dict(dy=0)]), NULL, "dy"), (dict(tensors=[dict(dx=0)]), NULL, "dx"),
    (dict(tensors=[dict(dy=P + 1)]), ALIGN, "dy"), (dict(tensors=[dict(dw=P + 1)]), ALIGN, "dweight"),
    (dict(tensors=[dict(w=0)]), NULL, "without weight"), (dict(ws=0), NULL, "ws"), (dict(ws=16 * P + 8), ALIGN, "ws"),
    (dict(nb=16), SHAPE, "ws_bytes=16"), (dict(tensors=[dict(dx=P, yt=256)]), UNSUP, "in place"),
    (dict(tensors=[dict(dx=2 * P, yh=128, yt=256)]), UNSUP, "in place"), (dict(tensors=[dict(dx=4 * P)]), UNSUP, "weight"),
    (dict(tensors=[dict(dw=4 * P)]), UNSUP, "weight"), (dict(tensors=[dict(dw=4 * P + 126)]), UNSUP, "weight"),
    (dict(tensors=[dict(dw=P)]), UNSUP, "dweight"), (dict(tensors=[dict(dw=16 * P)]), UNSUP, "ws"),
    (dict(ws=P), UNSUP, "ws"), (dict(ws=4 * P), UNSUP, "ws"),
    (dict(tensors=[{}, dict(x=6 * P, dy=7 * P)]), UNSUP, "one buffer"),
    (dict(tensors=[{}, dict(x=6 * P, dy=7 * P, dx=2 * P, dw=9 * P)]), UNSUP, "tensors[0].dy"),
    (dict(tensors=[{}, dict(x=6 * P, dy=7 * P, dx=8 * P)]), UNSUP, "another dweight")])
def test_backward_refusals(q, kw, status, text):
    assert bwd(q, **kw) == status, q.last_error()
    assert text in q.last_error()


def test_workspace(q):
    for T, D, heads in ((1, 64, (32, 4)), (100000, 128, (32, 8)), (61, 80, (12,)), (5, 1024, (1, 1, 1, 1))):
        n = q.norm_rope_backward_bytes(T, D, *heads)
        assert n > 0 and n % (4 * D) == 0 and n <= 4 * D * (1024 + len(heads)), n
    out = ctypes.c_size_t(0)
    one = (ctypes.c_int64 * 1)(4)
    call = lambda *a: q.raw_call("qmv_norm_rope_backward_bytes", *a)  # noqa: E731
    assert call(0, 64, 1, one, ctypes.byref(out)) == SHAPE and call(1, 2000, 1, one, ctypes.byref(out)) == SHAPE
    assert call(1, 64, 0, one, ctypes.byref(out)) == SHAPE and call(1, 64, 1, None, ctypes.byref(out)) == NULL
    assert call(1, 64, 1, one, None) == NULL and call(1 << 31, 64, 1, one, ctypes.byref(out)) == OVER


def test_binding_refusals(q):
    """Shapes and types that the pointers cannot show (CPU tensors get no further than the device check)."""
    x, w, pos, f = torch.zeros(3, 2, 8), torch.zeros(8), torch.zeros(3, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError, match="live on the GPU"):
        q.norm_rope(x, None, w, None, pos, f)
    with pytest.raises(ValueError, match="expected \\[T\\]"):
        q.norm_rope(x[0], None, w, None, pos, f)
    with pytest.raises(ValueError, match="pos holds 2"):
        q.norm_rope(x, None, w, None, pos[:2], f)
    with pytest.raises(ValueError, match="k has shape"):
        q.norm_rope(x, x[:, :, :4], w, None, pos, f)
    with pytest.raises(ValueError, match="k_weight is given"):
        q.norm_rope(x, None, w, w, pos, f)
    with pytest.raises(ValueError, match="k_out is given"):
        q.norm_rope(x, None, w, None, pos, f, k_out=x)
    with pytest.raises(ValueError, match="unknown layout"):
        q.norm_rope(x, None, w, None, pos, f, layout="pairs")
    with pytest.raises(ValueError, match="go together"):
        q.norm_rope_backward(x, x, w, w, x, None, pos, f)
