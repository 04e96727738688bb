"""Buffers of the gated products that overlap in part: refused on the host.  64
tokens of 64 values take 8192 bytes."""
import pytest

UNSUP = -3
P = 1 << 20  # addresses that no refused call touches
N = K = M = 64
B = 2 * M * N


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


@pytest.mark.parametrize("x,h,g,u,text", [
    (1, 1 + 0.5, 4, 6, "H overlaps X"), (1, 0.5, 4, 6, "H overlaps X"), (1, 3, 3.5, 6, "G overlaps H"),
    (1, 3, 5, 4.25, "U overlaps G"), (1, 3, 5, 1.75, "U overlaps X"), (1, 3, 5, 2.5, "U overlaps H"),
    (1, 2 - 16 / B, None, None, "H overlaps X")])
def test_forward(q, x, h, g, u, text):
    x, h, g, u = (0 if v is None else P + int(v * B) for v in (x, h, g, u))
    assert q.raw_call("qmv_gemm_glu", 2, N, K, M, P, P, x, 3, 1, h, 3, g, u, None) == UNSUP
    assert q.last_error() == text


@pytest.mark.parametrize("kw,text", [
    (dict(dg=0.5), "dG overlaps G"), (dict(du=2.5), "dU overlaps U"), (dict(dg=6, du=6.5), "dU overlaps dG"),
    (dict(dx=4.5), "dX overlaps dH"), (dict(dx=6.5), "dX overlaps dG"), (dict(dg=0, du=2, dx=0.5), "dX overlaps G"),
    (dict(ws=4.5), "ws overlaps dH"), (dict(ws=10.5), "ws overlaps dX")])
def test_backward(q, kw, text):
    at = dict(g=0, u=2, dh=4, dg=6, du=8, dx=10, ws=100)
    at.update(kw)
    p = {k: P + int(v * B) for k, v in at.items()}
    need = q.gemm_glu_backward_bytes("w4a16_g64", N, K, M, unrounded=True)
    assert need >= 2 * B
    status = q.raw_call("qmv_gemm_glu_backward_ex", 2, N, K, M, P, P, p["g"], p["u"], p["dh"], 3, 1, 1, p["dg"], p["du"],
                        p["dx"], p["ws"], need, None)
    assert status == UNSUP and q.last_error() == text
