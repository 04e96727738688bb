"""Arguments of the rotary positions that a call would leave aside."""
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    import gemm_dequant_matvec_amd as mod
    return mod


def test_output_without_its_input(q):
    x, pos, f = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int64), torch.zeros(32)
    with pytest.raises(ValueError, match="k_out is given without k"):
        q.rope(x, None, pos, f, k_out=torch.zeros(4, 2, 64))
