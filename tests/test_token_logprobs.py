"""Log probabilities, entropy and likeliest tokens against their definitions in 64 bits.

Tolerances in units of U = 2^-24.  S1 and S2 are sums of terms of one sign: a term is
off by at most 8 U of it (the exponential's 4, its argument's rounding, at most 1.5 d,
times e^d, below 1), and a thread adds V / 256 of them at most before a hundred more
additions and products join the threads and CTAs: rel = (V / 256 + 110) U.  ln S1 is
off by rel and 2 U of itself, d by U |d|; S2 / S1 by 3 rel of itself.
"""
import ctypes
import math

import pytest
import torch

import selective_state_space_conv1d_gb300 as m

FAKE = ctypes.c_void_p(0x100000)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def reference(logits):
    """ln p, entropy, and ln S1 (for the bounds) in 64 bits; a row of -inf has neither NaN."""
    l = logits.cpu().double()
    top = l.amax(-1, keepdim=True)
    d = torch.where(l == -math.inf, l, l - top)
    e = torch.exp(d)
    s1 = e.sum(-1)
    lp = d - torch.log(s1)[:, None]
    lp = torch.where((l == -math.inf) & ~s1.isnan()[:, None], torch.full_like(lp, -math.inf), lp)
    h = -torch.where(e > 0, e * lp, torch.zeros_like(e)).sum(-1) / torch.where(s1 == 0, torch.ones_like(s1), s1)
    h = torch.where(s1.isnan(), s1, h)
    return lp, h, torch.log(s1)


def run(logits, tokens=None, n=0, entropy=True):
    M = logits.shape[0]
    new = lambda *s, dt=torch.float32: torch.full(s, -777, dtype=dt, device="cuda")  # noqa: E731
    lp = new(M) if tokens is not None else None
    h = new(M) if entropy else None
    tl, ti = (new(M, n), new(M, n, dt=torch.int64)) if n else (None, None)
    m.mamba_token_logprobs(lp, h, tl, ti, logits, tokens)
    return lp, h, tl, ti


def close(got, ref, tol, what):
    got = got.cpu().double()
    same = (got == ref) | (got.isnan() & ref.isnan())  # infinities and NaN in their places
    err = (got - ref).abs()
    ok = same | (err <= tol)
    assert bool(ok.all()), f"{what}: off by {(err / tol)[~ok].max():.3g} of the bound"


def check(logits, tokens, n):
    V = logits.shape[1]
    lp, h, tl, ti = run(logits, tokens, n)
    ref, ref_h, log_s1 = reference(logits)
    rel = (V / 256 + 110) * U
    bound = lambda x: rel + 4 * U * (log_s1.abs().reshape(x.shape[0], *[1] * (x.dim() - 1)) + x.abs())  # noqa: E731
    if tokens is not None:
        want = ref.gather(1, tokens.cpu()[:, None])[:, 0]
        close(lp, want, bound(want), "logprob")
    close(h, ref_h, rel + 4 * U * log_s1.abs() + 4 * rel * (ref_h - log_s1).abs(), "entropy")
    if n:
        order = torch.sort(logits.cpu(), dim=-1, descending=True, stable=True).indices[:, :n]
        assert torch.equal(ti.cpu(), order)
        want = ref.gather(1, order)
        close(tl, want, bound(want), "top")


# ------------------------------------------------------------------ refusals, on the CPU

def _call(**kw):
    far = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 9)]
    a = dict(lp=far[0], h=far[1], tl=far[2], ti=far[3], logits=far[4], ld=100, dt=1, tokens=far[5], n=4, M=4, V=100)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.load().mamba_token_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), -1), (dict(tokens=None), -1), (dict(lp=None), -1), (dict(tl=None), -1), (dict(ti=None), -1),
    (dict(n=0), -1), (dict(n=-1), -1), (dict(n=33), -2), (dict(n=5, V=4, ld=4), -1), (dict(dt=2), -1), (dict(ld=99), -1),
    (dict(M=-1), -1), (dict(V=0), -1), (dict(V=1 << 31, ld=1 << 31), -1), (dict(M=1 << 40), -1), (dict(lp=FAKE, h=FAKE), -1),
    (dict(lp=FAKE, logits=FAKE), -1), (dict(ti=FAKE, tokens=FAKE), -1), (dict(tl=FAKE, ti=FAKE), -1),
    (dict(logits=ctypes.c_void_p(0x5000001)), -1), (dict(ti=ctypes.c_void_p(0x4000004)), -1),
])
def test_refusals(kw, code):
    assert _call(**kw) == code
    assert m.mamba_last_error()


def test_empty_and_partial_calls_pass_the_host_checks():
    assert _call(M=0) == 0
    for kw in (dict(tokens=None, lp=None), dict(n=0, tl=None, ti=None), dict(h=None)):
        assert _call(**kw) != 0 and "go" not in m.mamba_last_error().split(), m.mamba_last_error()


def test_python_refusals():
    l, f, i = torch.zeros(3, 50), torch.zeros(3), torch.zeros(3, dtype=torch.int64)
    tl, ti = torch.zeros(3, 4), torch.zeros(3, 4, dtype=torch.int64)
    good = dict(logprob=f, entropy=f.clone(), top_logprob=tl, top_id=ti, logits=l, tokens=i)
    for kw in (dict(logits=l[0]), dict(logits=l.half()), dict(tokens=i.int()), dict(tokens=i[:2]), dict(logprob=f[:2]),
               dict(logprob=f.double()), dict(entropy=f[:1]), dict(top_id=None), dict(top_logprob=None),
               dict(top_id=ti.int()), dict(top_id=ti[:, :3]), dict(top_id=ti[0]), dict(top_logprob=tl[:2]),
               dict(logits=l.T.contiguous().T)):
        with pytest.raises((ValueError, TypeError)):
            m.mamba_token_logprobs(*{**good, **kw}.values())


# ------------------------------------------------------------------ on the GPU

def rows(seed, M, V, dtype="f32", spread=3.0):
    g = torch.Generator().manual_seed(seed)
    l = (spread * torch.randn(M, V, generator=g)).to(DT[dtype]).cuda()
    return l, torch.randint(0, V, (M,), generator=g).cuda()


SIZES = [1, 2, 3, 8, 9, 31, 100, 255, 256, 257, 1000, 1500, 2047, 2048, 2049, 4099, 8191, 16384, 32003, 50000, 131072,
         262147]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", SIZES)
def test_vocabularies(cuda_lib, V, dtype):
    """bf16 logits of a large vocabulary hold many equal values: the lowest index first."""
    l, t = rows(V, 5, V, dtype)
    for n in {0, 1, min(5, V), min(32, V)}:
        check(l, t, n)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 19, 38, 39, 76, 77, 152, 153, 305, 1200])
def test_rows(cuda_lib, M):
    l, t = rows(M, M, 9001, "bf16")
    check(l, t, 7)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 1000, 40001])
@pytest.mark.parametrize("keep", [0, 1, 3, 40])
def test_masked_rows(cuda_lib, V, dtype, keep):
    """Rows whose mask (of -inf, or of the type's lowest value) leaves `keep` tokens, or none."""
    for fill in (-math.inf, torch.finfo(DT[dtype]).min):
        l, t = rows(keep, 4, V, dtype)
        kept = torch.rand(4, V, generator=torch.Generator().manual_seed(3)).topk(keep).indices.cuda()
        masked = torch.full_like(l, fill).scatter(1, kept, l.gather(1, kept))
        if keep:
            t[:2] = kept[:2, 0]
        check(masked, t, 9)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [300, 20011])
def test_nan_and_infinity(cuda_lib, V):
    l, t = rows(1, 6, V)
    l[0, 17] = math.nan
    l[1, 200] = math.inf
    l[2] = -math.inf
    l[2, 40] = math.nan
    l[2, 41] = -math.nan
    l[3, 100:105] = 0.0
    l[3, 104] = -0.0
    l[3] = torch.where(l[3] > 0, -l[3], l[3])
    l[4, 11] = 3e38
    l[4, 12] = -3e38
    lp, h, tl, ti = run(l, t, 5)
    for i in (0, 1, 2):
        assert bool(lp[i].isnan() and h[i].isnan() and tl[i].isnan().all())
    assert ti[0, 0] == 17 and ti[1, 0] == 200 and ti[2, :2].tolist() == [40, 41] and ti[2, 2:].tolist() == [0, 1, 2]
    assert ti[3].tolist() == [100, 101, 102, 103, 104]
    check(l[3:], t[3:], 5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5000, 65536])
def test_equal_logits_and_values_that_repeat(cuda_lib, V, dtype):
    """All equal; rising; falling; the large values in one thread's vectors (more than the list of candidates holds)."""
    l, t = rows(2, 5, V, dtype)
    l[0] = 1.25
    ramp = torch.arange(V, device="cuda").float()
    l[1] = (ramp / 64).to(DT[dtype])
    l[2] = (-ramp / 64).to(DT[dtype])
    vec = 16 // l.element_size()
    mine = (torch.arange(V, device="cuda") // vec) % 256 < 40
    l[3] = torch.where(mine, 5 + (ramp % 7) / 8, l[3].float() - 20).to(DT[dtype])
    l[4, V // 2:] = 9.0
    check(l, t, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_alignment_and_partial_calls(cuda_lib, dtype):
    M, V = 7, 1003
    l, t = rows(3, M, V, dtype)
    want = run(l, t, 6)
    for off in (0, 1, 3, 8):
        wide = torch.full((M, V + 13), math.nan, dtype=DT[dtype], device="cuda")
        wide[:, off:off + V] = l
        check(wide[:, off:off + V], t, 6)
    lp, h, tl, ti = run(l, t, 0, entropy=False)
    assert torch.equal(lp, want[0]) and h is None
    lp, h, tl, ti = run(l, None, 6)
    assert lp is None and torch.equal(h, want[1]) and torch.equal(tl, want[2]) and torch.equal(ti, want[3])
    m.mamba_token_logprobs(None, None, None, None, l)


@pytest.mark.gpu
def test_padding_and_tokens_outside(cuda_lib):
    l, t = rows(4, 6, 777)
    want = run(l, t)[0]
    t[1], t[3], t[4], t[5] = -1, -100, 777, 1 << 40
    lp = run(l, t)[0]
    assert torch.equal(lp[[0, 2]], want[[0, 2]]) and lp[1] == 0 and lp[3] == 0 and bool(lp[4:].isnan().all())


@pytest.mark.gpu
def test_a_large_call_past_32_bits(cuda_lib):
    """Rows past 2^31 elements from the first."""
    M, V = 17000, 131072
    l = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    t = torch.arange(M, device="cuda") * 7 % V
    l[torch.arange(M, device="cuda"), t] = 8.0
    lp, h, tl, ti = run(l, t, 2)
    p = math.exp(8) / (math.exp(8) + V - 1)
    assert torch.equal(ti[:, 0], t) and torch.equal(ti[:, 1], (t == 0).long())
    assert float((lp.double() - math.log(p)).abs().max()) < (V / 256 + 200) * U
    want = -p * math.log(p) - (1 - p) * math.log((1 - p) / (V - 1))
    assert float((h.double() - want).abs().max()) < 20 * (V / 256 + 200) * U


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 400])
def test_on_another_stream_and_in_a_graph(cuda_lib, M):
    l, t = rows(5, M, 30000, "bf16")
    outs = run(l, t, 8)
    want = [o.clone() for o in outs]
    st = torch.cuda.Stream()
    for o in outs:
        o.zero_()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        m.mamba_token_logprobs(*outs, l, t)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mamba_token_logprobs(*outs, l, t)
    for o in outs:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 30011])
@pytest.mark.parametrize("offset", [1e5, -1e5, 1e8, -1e9, -1e20, 1e30, -3e38])
def test_rows_far_from_zero_and_masks_of_any_size(cuda_lib, V, dtype, offset):
    """Rows of one far value, and rows of ordinary ones among far ones."""
    l, t = rows(6, 4, V, dtype)
    l[0] = offset
    l[1, ::3] = offset
    l[2] = torch.where(torch.arange(V, device="cuda") % 5 == 0, l[2].float(), -abs(offset)).to(DT[dtype])
    l[3, V // 2:] = offset
    # ln p of a token is as exact as its difference from the maximum, which the reference takes from the same logits
    check(l, t, 6)


@pytest.mark.gpu
def test_steep_rows(cuda_lib):
    """Differences of hundreds: every part but the largest underflows."""
    l, t = rows(7, 5, 50000, "f32", spread=300.0)
    check(l, t, 12)
