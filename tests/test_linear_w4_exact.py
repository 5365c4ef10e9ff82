"""Projections with 4-bit weights whose sums are exact in 32 bits, compared for equality.

Activations are whole numbers up to 3 and scales 1/2, 1, 2 or 4, so every term is a
multiple of 1/2, and every sum of them, in any order, is at most 3 * 15 * 4 K in size: up
to K = 46603 fewer than 2^24 halves.  A scale or a zero point of a wrong group
then shows at any K; the few-row kernels hold the scales of 8192 k at once.
"""
import pytest
import torch

import selective_state_space_conv1d_gb300 as m


def inputs(seed, M, N, K, group, zeros, scales=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda")  # noqa: E731
    G = -(-K // group)
    q = new(0, 256, N, -(-K // 32) * 16).to(torch.uint8)
    s = torch.exp2(new(-1, 3, N, G).float()).to(scales)
    z = new(0, 16, N, G).to(torch.uint8) if zeros else None
    a = torch.nn.functional.pad(new(-3, 4, M, K), (0, -K % 8)).to(torch.bfloat16)[:, :K]
    return a, q, s, z


def exact(a, q, s, z, group):
    K = a.shape[1]
    spread = lambda t: t.double().repeat_interleave(group, 1)[:, :K]  # noqa: E731
    v = torch.stack((q & 15, q >> 4), -1).flatten(1)[:, :K].double()
    return a.double() @ ((v - (8 if z is None else spread(z))) * spread(s)).T


def compare(a, q, s, z, group, rows=slice(None)):
    c = torch.full((a.shape[0], q.shape[0]), float("nan"), device="cuda")
    m.mamba_linear_w4(c, a, q, s, z, group=group)
    want = exact(a, q[rows], s[rows], None if z is None else z[rows], group)
    assert torch.equal(c[:, rows].double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 40, 130, 200])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [8192, 8200, 16384 + 40, 32768 + 40])
def test_many_spans_of_scales(cuda_lib, K, group, M):
    for zeros in (False, True):
        compare(*inputs(K + M, M, 45, K, group, zeros, torch.float32 if M % 2 else torch.bfloat16), group)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 8])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", [9751, 19467, 38939])
def test_many_spans_by_few_warps_a_row(cuda_lib, N, group, M):
    """So many weight rows that eight, four or two warps share 16 of them, past their first span."""
    K = 8192 + 1000
    args = inputs(N + M, M, N, K, group, True)
    compare(*args, group, torch.cat((torch.arange(0, N, 97), torch.arange(N - 33, N))))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 8, 24, 100, 193])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 40), (17, 127), (129, 129), (300, 416), (272, 2600)])
def test_ragged_sizes(cuda_lib, N, K, group, M):
    for zeros in (False, True):
        compare(*inputs(N, M, N, K, group, zeros), group)
