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


# Error of f32 results in the mean.  A value is a sum of up to dk + 128 products (over the key components and over two
# chunks' tokens), whose additions' and operands' errors of at most 2^-24 are independent: their root mean square is
# at most sqrt(dk + 128) 2^-24 of the values', and keys of unit length make the rule a contraction, so errors of earlier
# chunks do not grow.  (Sixteen bits in one operand are 2^-18 of it, four times this and more.)
def check_rms(x, y, s):
    ry, rs, _, _ = base.reference(x)
    tol = (x["q"].shape[3] + 128) ** 0.5 * 2.0 ** -24
    for what, got, ref in (("y", y, ry), ("state", s, rs)):
        err = (got.cpu().double() - ref).square().mean().sqrt() / ref.square().mean().sqrt()
        assert err <= tol, f"{what}: relative error {err:.2e}, allowed {tol:.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv", [
    (2, 16, 2, 4, 128, 128), (2, 17, 2, 4, 128, 128), (2, 200, 2, 4, 128, 128), (2, 17, 2, 2, 64, 64), (2, 200, 1, 2, 64, 64),
    (1, 200, 1, 2, 96, 200), (1, 150, 2, 2, 72, 40), (1, 200, 1, 1, 200, 64), (1, 130, 1, 2, 100, 130),
    (1, 2048, 1, 2, 128, 128), (1, 1500, 2, 2, 64, 128), (1, 200, 170, 170, 128, 64), (2, 100, 80, 80, 64, 64),
])
def test_f32_outputs_keep_32_bits(cuda_lib, B, T, Hk, Hv, dk, dv, dtype):
    x = base.make(91, B, T, Hk, Hv, dk, dv, dtype, device="cuda")
    x["dt_bias"] -= 2
    y, s = base.run_prefill(x, y_dtype=torch.float32)
    check_rms(x, y, s)


@pytest.mark.gpu
def test_the_type_of_y_changes_the_last_rounding_alone(cuda_lib):
    """Of the f32 and the bf16 output, the latter is off by half a step at most, and both leave one state."""
    for dk in (64, 128):
        x = base.make(92, 1, 300, 2, 2, dk, 128, "bf16", device="cuda")
        y, s = base.run_prefill(x)
        y32, s32 = base.run_prefill(x, y_dtype=torch.float32)
        assert torch.equal(s, s32)
        # half a step, and 2^-16 of the largest term for the products that a bf16 y may do without
        _, _, my, _ = base.reference(x)
        tol = 2.0 ** -8 * y32.cpu().double().abs() + 2.0 ** -16 * my[:, None, :, None]
        assert bool(((y.cpu().double() - y32.cpu().double()).abs() <= tol).all())


@pytest.mark.parametrize("dk,dv", [(0, 8), (8, 0), (0, 0)])
def test_heads_of_no_components_are_refused_by_the_library(dk, dv):
    x = base.make(0, 2, 5, 2, 4, max(dk, 1), max(dv, 1))
    q, v, s = x["q"][..., :dk], x["v"][..., :dv], torch.zeros(1, 2, 4, dv, dk)
    with pytest.raises(m.MambaError):
        m.mamba_gated_delta_prefill(v.clone(), q, q, v, x["a"], x["b"], x["A_log"], x["dt_bias"], None, s[0], stream=0)
    one = [t[:, 0].contiguous() for t in (v, q, q, v, x["a"], x["b"])]
    with pytest.raises(m.MambaError):
        m.mamba_gated_delta_step_batched(*one, x["A_log"], x["dt_bias"], s, 0, stream=0)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,Hv,T,dk,dv,dtype", [
    (2, 90, 90, 200, 64, 64, "bf16"), (1, 100, 200, 70, 128, 128, "bf16"), (1, 40, 80, 150, 128, 200, "bf16"),
    (2, 80, 80, 140, 64, 64, "f32"), (1, 160, 160, 65, 96, 72, "f32"),
])
def test_hand_overs_with_the_state_in_place(cuda_lib, B, Hk, Hv, T, dk, dv, dtype):
    """More items than SMs: one begins on an SM and ends on the next, which writes the state it began from."""
    assert m.mamba_gated_delta_workspace_bytes(B, T, Hk, Hv, dk, dv, 1 if dtype == "bf16" else 0) > 0
    x = base.make(101, B, T, Hk, Hv, dk, dv, dtype, device="cuda")
    x["dt_bias"] -= 3
    y, s = base.run_prefill(x)
    base.check(x, y, s)
    for _ in range(3):
        y1, s1 = base.run_prefill(x, inplace=True)
        assert torch.equal(y, y1) and torch.equal(s, s1)
    assert m.mamba_device_faults() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_y_far_apart(cuda_lib, dtype):
    """A row stride past the chunked kernel's 32-bit offsets."""
    x = base.make(102, 1, 40, 1, 2, 64, 32, dtype, device="cuda")
    ld = 1 << 23
    buf = torch.zeros(39 * ld + 64, dtype=base.DT[dtype], device="cuda")
    y = buf.as_strided((1, 40, 2, 32), (40 * ld, ld, 32, 1))
    s = torch.empty(1, 2, 32, 64, device="cuda")
    m.mamba_gated_delta_prefill(y, x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"], x["state_in"], s)
    torch.cuda.synchronize()
    base.check(x, y, s)
    assert int(buf.count_nonzero()) <= y.numel()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinity_leaves_the_groups_before_it(cuda_lib, dtype):
    x = base.make(103, 1, 300, 1, 2, 64, 64, dtype, device="cuda")
    y0, s0 = base.run_prefill(x)
    x["v"][0, 100, 0, 3] = float("inf")
    x["v"][0, 213, 0, 9] = -float("inf")
    y, s = base.run_prefill(x)
    others = [n for n in range(64) if n not in (3, 9)]
    assert torch.equal(y[:, :, 1], y0[:, :, 1]) and torch.equal(s[:, 1], s0[:, 1])
    assert torch.equal(y[..., others], y0[..., others]) and torch.equal(s[:, :, others], s0[:, :, others])
    for n, t in ((3, 100), (9, 213)):
        assert torch.equal(y[0, :t // 16 * 16, 0, n], y0[0, :t // 16 * 16, 0, n])
        assert not bool(torch.isfinite(y[0, t:, 0, n]).any()) and not bool(torch.isfinite(s[0, 0, n]).any())


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,Hv,T,dk,dv,dtype", [
    (1, 48, 48, 1280, 128, 128, "f32"), (1, 2, 4, 700, 128, 128, "f32"), (1, 12, 12, 740, 64, 64, "f32"),
    (1, 1, 1, 400, 72, 40, "f32"), (1, 2, 4, 760, 64, 64, "bf16"),
])
def test_sequences_that_are_cut_by_their_own_type_s_times(cuda_lib, B, Hk, Hv, T, dk, dv, dtype):
    """A chunk of f32 tensors takes two to three times one of bf16: shorter sequences of them are worth cutting."""
    assert m.mamba_gated_delta_workspace_bytes(B, T, Hk, Hv, dk, dv, 1 if dtype == "bf16" else 0) > 0
    x = base.make(104, B, T, Hk, Hv, dk, dv, dtype, device="cuda")
    x["dt_bias"] -= 4
    y, s = base.run_prefill(x)
    base.check(x, y, s)
    if dtype == "f32":
        check_rms(x, y, s)
