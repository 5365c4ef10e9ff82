"""Weights of 4 bits, as mamba_linear_w4 and the block calls take them.

A weight [N, K] is scales[n, k // group] * (q[n, k] - zeros[n, k // group]) with q in
0..15; a row of q is stored in ceil(K / 32) * 16 bytes, byte j holding k = 2j in its low
half and 2j + 1 in its high half.  Weights are made once, on any device, before they are
used; what a quantiser of a user's own makes is packed with pack_w4.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

GROUPS = (32, 64, 128)


class W4(NamedTuple):
    """A weight [N, K]: q uint8 [N, ceil(K / 32) * 16], scales f32 or bf16 [N, ceil(K /
    group)], zeros uint8 of that shape, 0..127 (None: 8)."""
    q: torch.Tensor
    scales: torch.Tensor
    zeros: Optional[torch.Tensor] = None
    group: int = 128


def pack_w4(values):
    """The stored rows of q: values [N, K] of 0..15 (any integer dtype) -> uint8."""
    if values.dim() != 2 or values.is_floating_point():
        raise ValueError("values must be an integer [N, K] tensor")
    if values.numel() and (int(values.min()) < 0 or int(values.max()) > 15):
        raise ValueError("values must be in 0..15")
    K = values.shape[1]
    v = torch.nn.functional.pad(values.to(torch.uint8), (0, -K % 32))
    return v[:, 0::2] | v[:, 1::2] << 4


def unpack_w4(q, K):
    """The values [N, K] of stored rows."""
    return torch.stack((q & 15, q >> 4), -1).flatten(1)[:, :K]


def quantize_w4(weight, group=128, *, zeros=False, scale_dtype=torch.bfloat16):
    """A floating-point weight [N, K] to the nearest 4-bit one, group by group: values -7..7
    of a scale max|w| / 7, or, with zeros, 0..15 of a scale (max - min) / 15 with a zero
    point (max and min of the group and 0).  Weights have to be finite, and so has a
    group's max - min in f32."""
    if weight.dim() != 2 or not weight.is_floating_point():
        raise ValueError("weight must be a floating-point [N, K] tensor")
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group}")
    if scale_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"scale_dtype must be float32 or bfloat16, got {scale_dtype}")
    N, K = weight.shape
    p = torch.nn.functional.pad(weight.float(), (0, -K % group)).view(N, -(-K // group), group)
    tiny = torch.finfo(torch.float32).tiny * 256  # a group of zeros keeps a scale
    if zeros:
        lo, hi = p.amin(-1).clamp(max=0), p.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).clamp(min=tiny).to(scale_dtype)
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s = (p.abs().amax(-1) / 7).clamp(min=tiny).to(scale_dtype)
        z = torch.full_like(s, 8, dtype=torch.float32)
    if not bool(s.isfinite().all()):
        raise ValueError("weight must be finite, and so must each group's range in float32")
    v = (torch.round(p / s.float()[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8)
    return W4(pack_w4(v.flatten(1)[:, :K]), s, z.to(torch.uint8) if zeros else None, group)


def dequantize_w4(w, K):
    """The weight [N, K] of a W4, in f32."""
    spread = lambda t: t.float().repeat_interleave(w.group, 1)[:, :K]  # noqa: E731
    return (unpack_w4(w.q, K).float() - (8.0 if w.zeros is None else spread(w.zeros))) * spread(w.scales)
