"""The gated delta rule where the forms of a call differ: ragged ends, hand-overs,
strides, output types.  Against the recurrence in 64 bits.
"""
import importlib.util
import os

import pytest
import torch

import selective_state_space_conv1d_gb300 as m

_spec = importlib.util.spec_from_file_location("gated_delta_cases", os.path.join(os.path.dirname(__file__),
                                                                                 "test_gated_delta.py"))
base = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(base)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["A_log", "dt_bias"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [10, 17, 64, 100, 150])
def test_a_head_that_keeps_nothing(cuda_lib, T, dtype, name):
    """exp(A_log) past f32's range, or a bias of infinity: alpha = 0 at every token, and nothing of it at the tokens
    that fill the last chunk."""
    x = base.make(81, 2, T, 2, 2, 64, 64, dtype, device="cuda")
    x[name][1] = 100.0 if name == "A_log" else float("inf")
    y, s = base.run_prefill(x)
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(s).all())
    base.check(x, y, s)
