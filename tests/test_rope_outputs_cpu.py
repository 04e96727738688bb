"""Outputs of the rotary positions whose values lie on one another: refused on the
host, by strides of 4 tokens and 2 heads of 64 values."""
import pytest

UNSUP, SHAPE = -3, -4
P = 0x10000  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


def rope(q, T, heads, token, head, R=64):
    arr = (q.QmvRopeTensor * 1)()
    t = arr[0]
    t.x, t.y, t.heads, t.x_token, t.x_head, t.y_token, t.y_head = P, 2 * P, heads, 128, 64, token, head
    return q.raw_call("qmv_rope", T, 64, R, 1, 1, arr, 3, P, P, 1.0, 0, None)


@pytest.mark.parametrize("T,heads,token,head", [
    (4, 2, 0, 64), (4, 2, 128, 0), (4, 2, 128, 32), (4, 2, 64, 64), (4, 2, 100, 64), (4, 2, 127, 64), (4, 2, 64, 200),
    (4, 2, 1, 64), (4, 1, 63, 0), (1, 2, 0, 63), (4, 2, -64, 64), (4, 2, 128, -63), (4, 2, 64, 255), (2, 1 << 20, 1 << 25, 64)])
def test_values_on_one_another(q, T, heads, token, head):
    assert rope(q, T, heads, token, head) == UNSUP and "more than once" in q.last_error()
