"""The gated head norm at sizes where its loops and offsets change, against the
formula in 64 bits.

Tolerance in units of 2^-24 of the value, as for the small sizes: d / 2 for the
sum of d squares, 4 for the reciprocal square root, 4 for the products, 16 for
SiLU.  A bf16 output adds half a step, 2^-8 of the value.
"""
import pytest
import torch

import selective_state_space_conv1d_gb300 as m

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(out, y, z, w, what):
    y, z = y.double(), z.double()
    ref = y / (y.square().mean(-1, keepdim=True) + 1e-5).sqrt() * z * torch.sigmoid(z)
    ref = ref if w is None else ref * w.double()
    tol = (y.shape[-1] / 2 + 24) * 2.0 ** -24 * ref.abs()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    assert bool(((out.double() - ref).abs() <= tol + 1e-37).all()), what


@pytest.mark.gpu
def test_a_row_of_more_than_2_to_the_31_values(cuda_lib):
    H, d = (1 << 24) + 9, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    part = 1 << 16
    y, z = (torch.empty(1, 1, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (y, z):
        for lo in range(0, H, part):
            t[0, 0, lo:lo + part].normal_(generator=g)
    out = torch.full_like(y, float("nan"))
    m.mamba_head_norm_gated(out, y, z)
    torch.cuda.synchronize()
    for lo in (0, H // 3, (1 << 24) - part, H - part):
        at = slice(lo, lo + part)
        check(out[0, 0, at], y[0, 0, at], z[0, 0, at], None, lo)
    assert not any(bool(out[0, 0, lo:lo + part].isnan().any()) for lo in range(0, H, part))


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H,d", [
    # heads of which every group of lanes takes eight: over 152 x 16 CTAs of 64 / (d / 8) groups
    (52001, 3, 64), (160001, 1, 64), (11201, 7, 128), (77853, 1, 128), (13001, 3, 256), (38913, 1, 200), (20013, 5, 88),
])
def test_heads_past_one_for_each_group(cuda_lib, rows, H, d, dtype, in_place):
    g = torch.Generator(device="cuda").manual_seed(d)
    # the head after the last, as a sentinel
    buf = torch.randn(rows * H * d + d, generator=g, device="cuda").to(DT[dtype])
    y = buf[:rows * H * d].view(1, rows, H, d)
    z = torch.randn(1, rows, H, d, generator=g, device="cuda").to(DT[dtype])
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    was, after = y.clone(), buf[rows * H * d:].clone()
    full = buf if in_place else torch.full_like(buf, 5.0)
    out = full[:rows * H * d].view(1, rows, H, d)
    m.mamba_head_norm_gated(out, y, z, w)
    torch.cuda.synchronize()
    part = 1 << 14
    for lo in range(0, rows, part):
        at = slice(lo, lo + part)
        check(out[0, at], was[0, at], z[0, at], w, lo)
    assert torch.equal(full[rows * H * d:], after if in_place else torch.full_like(after, 5.0))
    assert in_place or torch.equal(y, was)
