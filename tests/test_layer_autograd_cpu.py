"""The many-token operators record nothing for autograd: tensors that want a
gradient are refused where gradients are enabled (found before anything reaches
the device)."""
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


def calls(q, want):
    """Every call with one tensor after the other that requires a gradient."""
    W = torch.zeros(q.packed_bytes("w4a16_g64", 64, 128), dtype=torch.uint8)
    pos = torch.zeros(4, dtype=torch.int64)

    def t(*shape, g=False, dt=torch.bfloat16):
        return torch.zeros(shape, dtype=dt, requires_grad=g and want)

    yield lambda: q.gemm_glu("w4a16_g64", W, W, t(4, 128, g=True), 64, 128)
    yield lambda: q.gemm_glu("w4a16_g64", W, W, t(4, 128), 64, 128, H=t(4, 64, g=True))
    yield lambda: q.gemm_glu("w4a16_g64", W, W, t(4, 128), 64, 128, G=t(4, 64), U=t(4, 64, g=True))
    for i in range(3):
        yield lambda: q.gemm_glu_backward("w4a16_g64", W, W, *(t(4, 64, g=j == i) for j in range(3)), 64, 128)
    for kw in ({"dG": t(4, 64, g=True)}, {"dU": t(4, 64, g=True)}, {"dX": t(4, 128, g=True)}):
        yield lambda: q.gemm_glu_backward("w4a16_g64", W, W, t(4, 64), t(4, 64), t(4, 64), 64, 128, **kw)
    f = torch.zeros(32)
    yield lambda: q.rope(t(4, 2, 64, g=True), None, pos, f)
    yield lambda: q.rope(t(4, 2, 64), t(4, 1, 64, g=True), pos, f)
    yield lambda: q.rope(t(4, 2, 64), None, pos, t(32, g=True, dt=torch.float32))
    x = t(4, 2, 64, g=True)
    yield lambda: q.rope(x, None, pos, f, q_out=x)


def test_refused(q):
    n = 0
    for call in calls(q, True):
        n += 1
        with pytest.raises(ValueError, match="records no gradient"):
            call()
    assert n == 13


def test_taken_otherwise(q):
    """Without gradients enabled, or without a tensor that wants one, the calls go on
    (to the next check: the tensors are not on the GPU)."""
    for call in calls(q, False):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with torch.no_grad():
        for call in calls(q, True):
            with pytest.raises(ValueError, match="on the GPU"):
                call()


def test_inside_an_autograd_function(q):
    """A function of the caller's own may use them in its forward and backward."""
    W = torch.zeros(q.packed_bytes("w4a16_g64", 64, 128), dtype=torch.uint8)

    class Glu(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X):
            return q.gemm_glu("w4a16_g64", W, W, X, 64, 128)

    with pytest.raises(ValueError, match="on the GPU"):
        Glu.apply(torch.zeros(4, 128, dtype=torch.bfloat16, requires_grad=True))
