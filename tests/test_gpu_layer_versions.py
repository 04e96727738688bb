"""Tensors that a caller has the many-token operators write into count as changed
for autograd."""
import pytest
import torch

import workloads as wl
from gpu_helpers import pack_dev

pytestmark = pytest.mark.gpu


def test_versions(qmv):
    fmt, M, N, K = "w4a16_g64", 5, 64, 128
    W = pack_dev(qmv, fmt, wl.gen_weights(fmt, N, K, (71, 0, 0)))

    def new(*shape):
        return torch.randn(shape, device="cuda").bfloat16()

    def versions(*ts):
        return [t._version for t in ts]

    X, H, G, U = new(M, K), new(M, N), new(M, N), new(M, N)
    before = versions(X, W, H, G, U)
    qmv.gemm_glu(fmt, W, W, X, N, K, H=H)
    assert versions(X, W, H, G, U) == [before[0], before[1], before[2] + 1, before[3], before[4]]
    qmv.gemm_glu(fmt, W, W, X, N, K, H=H, G=G, U=U)
    assert versions(X, W, H, G, U) == [before[0], before[1], before[2] + 2, before[3] + 1, before[4] + 1]
    dH, dX, dU = new(M, N), new(M, K), new(M, N)
    before = versions(W, G, U, dH, dX, dU)
    qmv.gemm_glu_backward(fmt, W, W, G, U, dH, N, K, dG=G, dU=dU, dX=dX)
    assert versions(W, G, U, dH, dX, dU) == [before[0], before[1] + 1, before[2], before[3], before[4] + 1, before[5] + 1]
    with torch.inference_mode():  # tensors without a counter
        qmv.gemm_glu(fmt, W, W, X, N, K, H=new(M, N))


def test_backward_through_a_rotated_tensor(qmv):
    """A graph that saved q before q was rotated in place must not run on."""
    pos, f = torch.arange(6).cuda(), qmv.rope_freqs(32)
    w = torch.randn(6, 2, 32, device="cuda", requires_grad=True)
    q, k = torch.randn(6, 2, 32, device="cuda"), torch.randn(6, 1, 32, device="cuda")
    y = (w * q).sum()  # saves q
    vq, v = q._version, k._version
    with torch.no_grad():
        qmv.rope(q, k, pos, f)
        assert (q._version, k._version) == (vq, v)  # no output given: nothing changed
        qmv.rope(q, k, pos, f, q_out=q, k_out=k)
    assert k._version == v + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
