"""The key / value cache and its attention without a GPU: exports, every refusal
(found on the host, before any launch), sizes."""
import ctypes
import os
import re
import struct

import pytest
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qmv_cache.h")
OK, NULL, FORMAT, UNSUP, SHAPE, ALIGN, DTYPE, OVER = 0, -1, -2, -3, -4, -5, -6, -7
P = 0x1000000  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


def test_exports(q):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(qmv_[a-z0-9_]+)\s*\(", text))
    lib = ctypes.CDLL(q.LIB_PATH)
    assert names == set(q.CACHE_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def cache(**kw):
    a = dict(fmt=1, page=16, pages=8, heads=2, D=64, data=P)
    a.update({k: v for k, v in kw.items() if k in a})
    return struct.pack("2i4q", *a.values())


def batch(**kw):
    a = dict(T=4, B=2, q_start=2 * P, kv_len=2 * P, table=2 * P, columns=3, stride=3)
    a.update({k: v for k, v in kw.items() if k in a})
    return struct.pack("7q", *a.values())


def args(**kw):
    a = dict(q=3 * P, out=4 * P, lse=0, q_heads=4, qt=256, qh=64, ot=256, oh=64, dtype=3, scale=1.0, window=0, prefix=0, max_q=1,
             max_kv=40)
    a.update({k: v for k, v in kw.items() if k in a})
    return struct.pack("8qif4q", *a.values())


SHARED = [(dict(cache=None), NULL, "cache"), (dict(fmt=2), FORMAT, "fmt=2"), (dict(page=0), SHAPE, "page=0"),
          (dict(page=24), SHAPE, "page=24"), (dict(page=1040), SHAPE, "page=1040"), (dict(D=0), SHAPE, "D=0"),
          (dict(D=48), SHAPE, "D=48"), (dict(D=288), SHAPE, "D=288"), (dict(heads=0), SHAPE, "heads=0"),
          (dict(pages=0), SHAPE, "pages=0"), (dict(heads=65536), OVER, "heads"), (dict(pages=1 << 31), OVER, "pages"),
          (dict(pages=2 ** 31 - 1, heads=65535), OVER, "2^50")]
CALLS = [(dict(data=0), NULL, "data"), (dict(data=P + 8), ALIGN, "data"), (dict(batch=None), NULL, "batch"),
         (dict(T=0), SHAPE, "T=0"), (dict(B=0), SHAPE, "B=0"), (dict(columns=0), SHAPE, "columns=0"),
         (dict(T=1 << 31), OVER, "T"), (dict(B=1 << 23), OVER, "2^23"), (dict(columns=1 << 27), OVER, "2^30"),
         (dict(stride=2), SHAPE, "stride=2"), (dict(q_start=0), NULL, "q_start"), (dict(kv_len=0), NULL, "kv_len"),
         (dict(table=0), NULL, "table"), (dict(table=P + 2), ALIGN, "table"), (dict(dtype=0), DTYPE, "dtype=0"),
         (dict(dtype=4), UNSUP, "f32")]


def kv(q, name, **kw):
    a = dict(k=3 * P, v=4 * P, kt=128, kh=64, vt=128, vh=64, dtype=3)
    a.update({k: v for k, v in kw.items() if k in a})
    return q.raw_call(name, None if "cache" in kw else cache(**kw), None if "batch" in kw else batch(**kw), a["k"], a["kt"],
                      a["kh"], a["v"], a["vt"], a["vh"], a["dtype"], None)


@pytest.mark.parametrize("kw,status,text", SHARED + CALLS + [
    (dict(k=0), NULL, "k is"), (dict(v=0), NULL, "v is"), (dict(k=P + 1), ALIGN, "k is"), (dict(v=3 * P + 1), ALIGN, "v is"),
    (dict(k=3 * P + 2, dtype=1), ALIGN, "k is"), (dict(k=P), UNSUP, "k lies"), (dict(v=P + 64), UNSUP, "v lies"), (dict(k=P - 64), UNSUP, "k lies"),
    (dict(v=P + (1 << 20), vt=-(1 << 19)), UNSUP, "v lies")])
def test_write_refusals(q, kw, status, text):
    assert kv(q, "qmv_kv_write", **kw) == status, q.last_error()
    assert text in q.last_error()


@pytest.mark.parametrize("kw,status,text", SHARED + CALLS + [
    (dict(k=0, v=0), NULL, "k and v"), (dict(k=3 * P, v=3 * P), UNSUP, "one buffer"), (dict(kt=64), UNSUP, "k holds"),
    (dict(vh=32), UNSUP, "v holds"), (dict(v=P + 64), UNSUP, "v lies")])
def test_read_refusals(q, kw, status, text):
    assert kv(q, "qmv_kv_read", **kw) == status, q.last_error()
    assert text in q.last_error()


def attend(lib, ws=8 * P, nb=1 << 24, **kw):
    return lib.raw_call("qmv_kv_attention", None if "cache" in kw else cache(**kw), None if "batch" in kw else batch(**kw),
                      None if "args" in kw else args(**kw), ws, nb, None)


@pytest.mark.parametrize("kw,status,text", SHARED + CALLS + [
    (dict(args=None), NULL, "args"), (dict(q_heads=0), SHAPE, "q_heads=0"), (dict(q_heads=3), SHAPE, "q_heads=3"),
    (dict(window=-1), SHAPE, "window"), (dict(prefix=-1), SHAPE, "prefix"), (dict(max_q=0), SHAPE, "max_q"),
    (dict(max_kv=0), SHAPE, "max_kv"), (dict(T=1 << 30, q_heads=4), OVER, "2^30"), (dict(q_heads=1 << 21), OVER, "q_heads"),
    (dict(q=0), NULL, "q is"), (dict(out=0), NULL, "out"), (dict(q=3 * P + 1), ALIGN, "q is"), (dict(out=4 * P + 1), ALIGN, "out"),
    (dict(lse=5 * P + 2), ALIGN, "lse"), (dict(scale=float("nan")), UNSUP, "scale"), (dict(scale=float("inf")), UNSUP, "scale"),
    (dict(out=3 * P, ot=512), UNSUP, "other strides"), (dict(ot=128), UNSUP, "more than once"), (dict(out=P), UNSUP, "in the cache"),
    (dict(lse=P), UNSUP, "in the cache"), (dict(lse=4 * P), UNSUP, "lse"), (dict(lse=3 * P), UNSUP, "lse"),
    (dict(prefix=16, ws=0), NULL, "ws"), (dict(prefix=16, ws=8 * P + 8), ALIGN, "ws"), (dict(prefix=16, nb=16), SHAPE, "ws_bytes=16"),
    (dict(prefix=16, ws=P), UNSUP, "cache"), (dict(out=P - 128), UNSUP, "in the cache"),
    (dict(lse=P - 16), UNSUP, "in the cache"), (dict(lse=4 * P + 512), UNSUP, "overlaps"), (dict(lse=3 * P - 32), UNSUP, "overlaps"),
    (dict(prefix=16, ws=3 * P + 64), UNSUP, "overlaps"), (dict(prefix=16, ws=4 * P - 16), UNSUP, "overlaps"),
    (dict(out=4 * P, ot=-256, lse=4 * P - 512), UNSUP, "overlaps"), (dict(qt=1 << 62, lse=3 * P + 4096), UNSUP, "overlaps"), (dict(prefix=16, ws=3 * P), UNSUP, "ws"), (dict(prefix=16, lse=8 * P), UNSUP, "lse")])
def test_attention_refusals(q, kw, status, text):
    assert attend(q, **kw) == status, q.last_error()
    assert text in q.last_error()


def test_sizes(q):
    out = ctypes.c_size_t(0)
    assert q.raw_call("qmv_kv_cache_bytes", cache(data=0), ctypes.byref(out)) == OK and out.value == 8 * 2 * 2 * (1024 + 64)
    assert q.raw_call("qmv_kv_cache_bytes", cache(fmt=5), ctypes.byref(out)) == OK and out.value == 8 * 2 * 2 * (512 + 64)
    assert q.raw_call("qmv_kv_cache_bytes", cache(), None) == NULL
    assert q.kv_cache_bytes("q4_0", 10, 4, 128, 64) == 10 * 4 * 4 * 4 * (512 + 64)
    n = lambda **kw: (q.raw_call("qmv_kv_attention_bytes", cache(**kw), batch(**kw), args(**kw), ctypes.byref(out)), out.value)  # noqa: E731
    assert n(max_kv=40, columns=3) == (OK, 0)  # one part: no scratch memory
    assert n(prefix=16)[1] > 0 and n(T=1, B=1, columns=1000, max_kv=16000)[1] > 0
    assert n(T=1 << 20, B=1 << 10, max_q=1 << 10) == (OK, 0)
    assert q.raw_call("qmv_kv_attention_bytes", cache(), batch(), args(), None) == NULL
    assert q.raw_call("qmv_kv_attention_bytes", cache(), batch(), args(max_kv=0), ctypes.byref(out)) == SHAPE


def test_binding_refusals(q):
    """Shapes and types that the pointers cannot show."""
    c = q.KVCache("q8_0", 4, 2, 32, 16, device="cpu")
    x, i = torch.zeros(3, 2, 32), lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="unknown cache format"):
        q.KVCache("q6k", 4, 2, 32)
    with pytest.raises(q.QmvError, match="D=33"):
        q.KVCache("q8_0", 4, 2, 33, device="cpu")
    with pytest.raises(ValueError, match="data holds 8 bytes"):
        q.KVCache("q8_0", 4, 2, 32, data=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="live on the GPU"):
        q.kv_write(c, x, x, i(1, 2), i(2), i(1))
    with pytest.raises(ValueError, match="k has shape"):
        q.kv_write(c, x[:, :1], x, i(1, 2), i(2), i(1))
    with pytest.raises(ValueError, match="live on the GPU"):
        q.kv_read(c, i(1, 2), i(2), i(1), 3)
    with pytest.raises(ValueError, match="q has shape"):
        q.kv_attention(c, x[:, :, :16], i(1, 2), i(2), i(1))
    with pytest.raises(ValueError, match="live on the GPU"):
        q.kv_attention(c, x, i(1, 2), i(2), i(1))
    with pytest.raises(ValueError, match="no sequences"):
        q._kv_batch(c, 3, c.data.get_device(), i(0, 2), i(1), i(0))
    with pytest.raises(ValueError, match="no pages"):
        q._kv_batch(c, 3, c.data.get_device(), i(1, 0), i(2), i(1))
    with pytest.raises(ValueError, match="records no gradient"):
        q.kv_attention(c, x.requires_grad_(), i(1, 2), i(2), i(1))
