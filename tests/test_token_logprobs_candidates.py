"""Rows with more candidates for the alternatives than the kernel's list holds: it then takes
one pass over the row per alternative, and the order of tokens is that of the list.

A row's large values lie in the vectors of a few threads, so fewer thread maxima than the
alternatives asked for are large, the bound falls below them, and every large value reaches
it.  How many do is counted here, on the host, for the row as the kernel cuts it.
"""
import math

import numpy as np
import pytest
import torch

import selective_state_space_conv1d_gb300 as m
from test_token_logprobs import DT, check, run

LIST = 2048     # candidates a CTA holds
THREADS = 256


def order_of(row):
    """The indexes of a row by value and then by index, NaN above all."""
    v = row.double().numpy()
    nan = np.isnan(v)
    return np.lexsort((np.arange(len(v)), -np.where(nan, 0, v), ~nan))


def candidates(row, skew, n, cluster, vec):
    """The most elements that reach the bound in any CTA's slice of a row whose first element
    is the `skew`-th of its 16-byte vector."""
    V = len(row)
    rank = np.empty(V, dtype=np.int64)
    rank[order_of(row)] = np.arange(V)
    at = (skew + np.arange(V)) // vec
    nv = (skew + V + vec - 1) // vec
    bounds, slices = [], []
    for c in range(cluster):
        lo, hi = nv * c // cluster, nv * (c + 1) // cluster
        inside = (at >= lo) & (at < hi)
        slices.append(rank[inside])
        best = np.full(THREADS, V)
        np.minimum.at(best, (at[inside] - lo) % THREADS, rank[inside])
        first = np.sort(best.reshape(-1, 32), 1)[:, :-(-n // 8) * 2].ravel()  # of each warp
        bounds.append(np.sort(first)[n - 1])
    return max(int((s <= min(bounds)).sum()) for s in slices)


def hot_rows(V, dtype, n_rows, seed=0):
    """Ordinary logits, large ones in the vectors of the first 40 threads."""
    g = torch.Generator().manual_seed(seed)
    vec = 16 // torch.tensor([], dtype=DT[dtype]).element_size()
    hot = (torch.arange(V) // vec) % THREADS < 40
    return torch.where(hot, 30.0, 0.0) + torch.randn(n_rows, V, generator=g)


def cluster_of(M, V):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = 1
    while c < 8 and M * c * 2 <= 2 * sms and V // (c * 2) >= 4096:
        c *= 2
    return c


def test_the_count_on_the_host():
    """Sixteen large thread maxima at most are seen of the first two warps': asking for more
    alternatives takes every large value in."""
    row = hot_rows(262147, "f32", 1)[0]
    large = int((row[:262144 // 8] > 15).sum())
    assert large == 5120 and candidates(row, 0, 32, 8, 4) >= large
    assert candidates(row, 0, 1, 8, 4) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("n", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V", [(5, 262147), (160, 65536)])
def test_more_candidates_than_the_list_holds(cuda_lib, M, V, dtype, n):
    base = hot_rows(V, dtype, 5)
    base[1, 0] = math.nan                     # the greatest key there is
    base[2, 0], base[2, 1], base[2, V - 1] = math.nan, math.inf, math.nan
    base[3, 7], base[3, V // 2] = math.inf, math.nan
    base[4, :3] = 60.0
    base = base.to(DT[dtype])
    l = base.repeat(M // 5, 1).cuda()
    cluster, vec = cluster_of(M, V), 16 // l.element_size()
    assert cluster == (8 if M == 5 else 1)
    for i in range(5):
        assert candidates(base[i], i * V % vec, n, cluster, vec) > LIST
    lp, h, tl, ti = run(l, torch.zeros(M, dtype=torch.int64, device="cuda"), n)
    for i in range(M):
        assert ti[i].tolist() == order_of(base[i % 5])[:n].tolist(), f"row {i}"
    nan = torch.tensor([i % 5 in (1, 2, 3) for i in range(M)], device="cuda")
    assert bool((tl.isnan().all(1) == nan).all()) and bool((lp.isnan() == nan).all()) and bool((h.isnan() == nan).all())
    sound = [0, 4] if M == 5 else [0, 4, M - 5, M - 1]
    check(l[sound], torch.full((len(sound),), 2, dtype=torch.int64, device="cuda"), n)
    assert m.mamba_device_faults() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 40, 5000, 262147])
def test_nan_first(cuda_lib, V):
    """A NaN at index 0 stands first, whatever follows."""
    g = torch.Generator().manual_seed(V)
    l = torch.randn(3, V, generator=g)
    l[:, 0] = math.nan
    l[1] = math.nan
    n = min(V, 32)
    ti = run(l.cuda(), None, n)[3].cpu()
    for i in range(3):
        assert ti[i].tolist() == order_of(l[i])[:n].tolist()
