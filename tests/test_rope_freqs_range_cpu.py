"""Bases whose frequencies f32 does not hold."""
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


@pytest.mark.parametrize("kw", [dict(R=64, base=1e-60), dict(R=4096, base=5e-324),
                                dict(R=8, base=1e300, scaling="ntk", factor=1e10), dict(R=4, scaling="ntk", factor=1e200)])
def test_refused(q, kw):
    with pytest.raises(q.QmvError) as e:
        q.rope_freqs(device="cpu", **kw)
    assert e.value.status == -3


@pytest.mark.parametrize("kw", [dict(R=2, base=1e-300), dict(R=64, base=1e-38), dict(R=4096, base=1e308),
                                dict(R=8, base=1e4, scaling="ntk", factor=1e20), dict(R=64, base=0.5, scaling="linear", factor=1e30)])
def test_finite(q, kw):
    f = q.rope_freqs(device="cpu", **kw)
    assert bool(torch.isfinite(f).all()) and bool((f >= 0).all())
