"""Outputs of the rotary positions in every order of strides that keeps values apart."""
import pytest
import torch

pytestmark = pytest.mark.gpu


# tokens around heads and heads around tokens, with and without room between; axes of one
@pytest.mark.parametrize("T,heads,token,head", [(4, 2, 128, 64), (4, 2, 200, 64), (4, 2, 64, 256), (4, 2, 192, 96),
                                                (4, 2, 70, 300), (4, 1, 64, 0), (4, 1, 64, 7), (1, 2, 0, 64), (1, 1, 0, 0)])
def test_values_apart(qmv, T, heads, token, head):
    x = torch.randn(T, heads, 64, device="cuda")
    pos, f = torch.arange(T).cuda() + 3, qmv.rope_freqs(40)
    base, _ = qmv.rope(x, None, pos, f)
    buf = torch.full((2048,), 7.0, device="cuda")
    y = buf.as_strided((T, heads, 64), (token, head, 1))
    out, _ = qmv.rope(x, None, pos, f, q_out=y)
    assert torch.equal(out, base)
    mask = torch.ones(2048, dtype=torch.bool, device="cuda")
    mask.as_strided((T, heads, 64), (token, head, 1)).fill_(False)
    assert bool((buf[mask] == 7.0).all())
