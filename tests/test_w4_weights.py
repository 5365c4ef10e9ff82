"""What quantize_w4 makes of weights that are no numbers, or too large for a scale."""
import math

import pytest
import torch

import selective_state_space_conv1d_gb300 as m


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [(0, 0), (2, 76)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64])
def test_weights_that_are_not_finite_are_refused(zeros, bad, at, dtype):
    w = torch.randn(3, 77).to(dtype)
    w[at] = bad
    for scale in (torch.float32, torch.bfloat16):
        with pytest.raises(ValueError, match="finite"):
            m.quantize_w4(w, 32, zeros=zeros, scale_dtype=scale)


@pytest.mark.parametrize("zeros", [False, True])
def test_weights_past_32_bits_are_refused(zeros):
    """Weights of 64 bits that are infinite in 32, and a range that is."""
    with pytest.raises(ValueError, match="finite"):
        m.quantize_w4(torch.tensor([[1e300, 1.0]], dtype=torch.float64), 32, zeros=zeros)
    wide = torch.tensor([[3e38, -3e38]])
    if zeros:
        with pytest.raises(ValueError, match="finite"):
            m.quantize_w4(wide, 32, zeros=True)
    else:
        assert m.unpack_w4(m.quantize_w4(wide, 32).q, 2).tolist() == [[15, 1]]


@pytest.mark.parametrize("zeros", [False, True])
def test_large_small_and_empty_weights_pass(zeros):
    for w in (torch.full((2, 40), 1e38), torch.full((2, 40), -1e-38), torch.zeros(0, 40), torch.zeros(2, 40)):
        q = m.quantize_w4(w, 32, zeros=zeros)
        assert bool(q.scales.isfinite().all()) and q.q.shape == (w.shape[0], 32)
