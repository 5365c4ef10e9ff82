"""Norms of queries and keys where the inputs are none: frequencies that are no numbers."""
import pytest
import torch

import selective_state_space_conv1d_gb300 as m


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 32), (128, 128), (50, 20)])
def test_a_frequency_that_is_no_number(cuda_lib, d, rot, interleaved, value):
    """cos and sin of position x NaN, and of infinity (position 0 too: 0 x infinity), are NaN: its pair is, the others
    are as before."""
    x = torch.randn(2, 5, 3, d, generator=torch.Generator().manual_seed(d)).cuda()
    freq = 10000.0 ** (-torch.arange(0, rot, 2).float() / rot)
    want, got = torch.empty_like(x), torch.empty_like(x)
    m.mamba_qk_norm_rotary(want, None, x, None, None, None, freq.cuda(), interleaved=interleaved)
    pair = 3
    freq[pair] = value
    m.mamba_qk_norm_rotary(got, None, x, None, None, None, freq.cuda(), interleaved=interleaved)
    at = [2 * pair, 2 * pair + 1] if interleaved else [pair, pair + rot // 2]
    rest = [c for c in range(d) if c not in at]
    assert bool(got[..., at].isnan().all())
    assert torch.equal(got[..., rest], want[..., rest])
