"""qmv_gemm_glu_backward_ex without a GPU: flags, refusals, workspace sizes."""
import ctypes

import pytest

OK, NULL, FORMAT, UNSUP, SHAPE, ALIGN = 0, -1, -2, -3, -4, -5
P = 0x10000  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


def back(q, flags, N=64, K=64, M=4, ws=0, nb=0, dx=6 * P, fmt=2):
    return q.raw_call("qmv_gemm_glu_backward_ex", fmt, N, K, M, P, P, P, 2 * P, 3 * P, 3, 1, flags, 4 * P, 5 * P, dx, ws,
                      nb, None)


def size(q, fmt, N, K, M, flags):
    out = ctypes.c_size_t()
    assert q.raw_call("qmv_gemm_glu_backward_ex_bytes", fmt, N, K, M, flags, ctypes.byref(out)) == OK, q.last_error()
    return out.value


def test_unknown_flags(q):
    for flags in (2, 3, -1, 1 << 30):
        assert back(q, flags) == UNSUP and "flag" in q.last_error()
        out = ctypes.c_size_t()
        assert q.raw_call("qmv_gemm_glu_backward_ex_bytes", 2, 64, 64, 4, flags, ctypes.byref(out)) == UNSUP


def test_refusals_of_the_call_without_flags(q):
    for flags in (0, q.GLU_UNROUNDED):
        assert back(q, flags, fmt=0) == FORMAT
        assert back(q, flags, K=32) == SHAPE
        assert back(q, flags, dx=0) == NULL and "dX" in q.last_error()
        assert back(q, flags, dx=P) == UNSUP and "dX is the buffer of G" in q.last_error()
        assert q.raw_call("qmv_gemm_glu_backward_ex_bytes", 2, 64, 64, 4, flags, None) == NULL


@pytest.mark.parametrize("fmt,N,K,M", [(2, 64, 64, 4), (2, 63, 64, 5), (3, 5632, 2048, 24), (8, 2731, 1024, 391)])
def test_workspace(q, fmt, N, K, M):
    """Without flags as before; unrounded: two more copies of rows of whole 16 bytes."""
    out = ctypes.c_size_t()
    assert q.raw_call("qmv_gemm_glu_backward_bytes", fmt, N, K, M, ctypes.byref(out)) == OK
    assert size(q, fmt, N, K, M, 0) == out.value == q.gemm_glu_backward_bytes(fmt, N, K, M)
    need = size(q, fmt, N, K, M, q.GLU_UNROUNDED)
    copies = 2 * M * (-(-N // 8) * 8) * 2
    assert need >= copies and (need - copies * (2 if N % 8 else 1)) % (4 * M * K) == 0  # the rest: partial sums
    assert need == q.gemm_glu_backward_bytes(fmt, N, K, M, unrounded=True)
    assert back(q, q.GLU_UNROUNDED, N, K, M, dx=1 << 30, fmt=fmt) == NULL and "ws" in q.last_error()
    assert back(q, q.GLU_UNROUNDED, N, K, M, dx=1 << 30, fmt=fmt, ws=1 << 34, nb=need - 1) == SHAPE
    assert str(need) in q.last_error()
    assert back(q, q.GLU_UNROUNDED, N, K, M, dx=1 << 30, fmt=fmt, ws=(1 << 34) + 8, nb=need) == ALIGN
