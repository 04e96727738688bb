"""Calls of the rotary positions that share buffers as they may."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_one_input_twice(qmv):
    """q and k may be one tensor where the outputs are two."""
    x = torch.randn(7, 2, 64, device="cuda")
    pos, f = torch.arange(7).cuda(), qmv.rope_freqs(64)
    base, _ = qmv.rope(x, None, pos, f)
    a, b = qmv.rope(x, x, pos, f)
    assert torch.equal(a, base) and torch.equal(b, base)


def test_neighbours_in_place(qmv):
    """Heads of q and k that lie in turn in one buffer, both in place."""
    x = torch.randn(9, 3, 2, 64, device="cuda")
    pos, f = torch.arange(9).cuda(), qmv.rope_freqs(48)
    base = [qmv.rope(x[:, :, i].contiguous(), None, pos, f)[0] for i in (0, 1)]
    qmv.rope(x[:, :, 0], x[:, :, 1], pos, f, q_out=x[:, :, 0], k_out=x[:, :, 1])
    for i in (0, 1):
        assert torch.equal(x[:, :, i], base[i])


def test_one_buffer_in_two_places(qmv):
    x, y = torch.randn(7, 2, 64, device="cuda"), torch.randn(7, 2, 64, device="cuda")
    pos, f = torch.arange(7).cuda(), qmv.rope_freqs(64)
    for kw in (dict(q_out=x, k_out=x), dict(q_out=y, k_out=x)):
        with pytest.raises(qmv.QmvError):
            qmv.rope(x, y, pos, f, **kw)
    with pytest.raises(qmv.QmvError):
        qmv.rope(x, x, pos, f, q_out=x, k_out=y)
