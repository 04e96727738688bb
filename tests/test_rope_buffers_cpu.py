"""Buffers that a call of the rotary positions would write while reading, or write
twice: refused on the host."""
import pytest

UNSUP = -3
P = 0x10000  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


def rope(q, *xy):
    arr = (q.QmvRopeTensor * len(xy))()
    for t, (x, y) in zip(arr, xy):
        t.x, t.y, t.heads, t.x_token, t.x_head, t.y_token, t.y_head = x * P, y * P, 2, 128, 64, 128, 64
    return q.raw_call("qmv_rope", 4, 64, 64, 1, len(xy), arr, 3, P, P, 1.0, 0, None)


@pytest.mark.parametrize("xy,text", [
    (((1, 1), (1, 1)), "tensors[0].y and tensors[1].y"),        # the same tensor twice, in place
    (((1, 2), (3, 2)), "tensors[0].y and tensors[1].y"),
    (((1, 3), (3, 4)), "tensors[0].y is the buffer of tensors[1].x"),
    (((3, 4), (1, 3)), "tensors[1].y is the buffer of tensors[0].x"),
    (((1, 2), (3, 3), (5, 6), (7, 5)), "tensors[3].y is the buffer of tensors[2].x")])
def test_one_buffer_in_two_places(q, xy, text):
    assert rope(q, *xy) == UNSUP and text in q.last_error()
