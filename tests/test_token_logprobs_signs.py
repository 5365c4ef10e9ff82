"""A log probability is at most 0 and an entropy at least 0, also where rounding would carry
them past it: rows of a certain token, and of one that is nearly so.

How far they may be off is that of test_token_logprobs.
"""
import math

import pytest
import torch

from test_token_logprobs import DT, check, rows, run


def certain_rows(M, V, dtype, below, seed=1):
    """Rows with a token of some size and the rest `below` under it (inf: masked)."""
    g = torch.Generator().manual_seed(seed)
    top = (30 * torch.randn(M, 1, generator=g)).to(DT[dtype]).float()
    t = torch.randint(0, V, (M,), generator=g)
    l = (top - below - torch.rand(M, V, generator=g)).scatter(1, t[:, None], top)
    return l.to(DT[dtype]).cuda(), t.cuda()


def signs(l, t, n):
    lp, h, tl, ti = run(l, t, n)
    for what, v, low in (("logprob", lp, False), ("entropy", h, True), ("top", tl, False)):
        wrong = v < 0 if low else v > 0
        assert not bool(wrong.any()), f"{what}: {int(wrong.sum())} of {v.numel()} past 0"
    return lp, h, tl, ti


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("below", [math.inf, 300.0, 40.0, 18.0])
@pytest.mark.parametrize("M,V", [(400, 1000), (400, 1), (30, 32003)])
def test_one_certain_token(cuda_lib, M, V, below, dtype):
    l, t = certain_rows(M, V, dtype, below)
    n = min(V, 3)
    lp, h, tl, ti = signs(l, t, n)
    assert torch.equal(ti[:, 0], t)
    check(l, t, n)
    # what a caller makes of them
    assert not bool((1 - lp.double().exp()).log().isnan().any()) and not bool(h.sqrt().isnan().any())


@pytest.mark.gpu
@pytest.mark.parametrize("far", [2.0 ** 24, -1e8, 3e38])
def test_far_rows(cuda_lib, far):
    l = torch.full((40, 3000), -math.inf).scatter(1, torch.arange(40)[:, None] * 70, far).cuda()
    t = torch.arange(40, device="cuda") * 70
    lp, h, tl, ti = signs(l, t, 1)
    assert not lp.any() and not h.any() and not tl.any()


@pytest.mark.gpu
def test_masked_rows_and_nan_keep_theirs(cuda_lib):
    l, t = rows(3, 5, 700)
    l[0] = -math.inf
    l[1, 5] = math.nan
    l[2, 6] = math.inf
    lp, h, tl, ti = run(l, t, 2)
    assert lp[0] == -math.inf and h[0] == 0 and bool((tl[0] == -math.inf).all())
    assert bool(lp[1:3].isnan().all() and h[1:3].isnan().all() and tl[1:3].isnan().all())
    assert bool((lp[3:] < 0).all() and (h[3:] > 0).all())
