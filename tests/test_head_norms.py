"""Per-head norms of queries and keys with the position rotation, and the gated
output norm, against their formulas in 64 bits.

Tolerance in units of 2^-24 of the value: d / 2 for the sum of d squares, 4 for
the reciprocal square root, 4 for the products; the rotation adds 16 of
|x| + |y| (an angle off by 2^-24 half-turns, and its sine and cosine), SiLU 16.
A bf16 output adds half a step, 2^-8 of the value.
"""
import ctypes

import pytest
import torch

import selective_state_space_conv1d_gb300 as m

FAKE = ctypes.c_void_p(0x100000)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def ref_norm(x, w, eps, l2):
    x = x.detach().cpu().double()
    ss = x.square().sum(-1, keepdim=True)
    x = x / torch.sqrt((ss if l2 else ss / x.shape[-1]) + eps)
    return x if w is None else x * w.cpu().double()


def ref_turn(x, inv_freq, positions, interleaved):
    """(turned, |x| + |y| of the pair) of the first components of x [B, T, H, d]."""
    if inv_freq is None:
        return x, x.abs()
    r = inv_freq.shape[0]
    th = (positions.cpu().double()[..., None] * inv_freq.cpu().double())[:, :, None]
    lo, hi = (x[..., 0:2 * r:2], x[..., 1:2 * r:2]) if interleaved else (x[..., :r], x[..., r:2 * r])
    a, b, size = lo * th.cos() - hi * th.sin(), hi * th.cos() + lo * th.sin(), lo.abs() + hi.abs()
    join = (lambda p, q: torch.stack((p, q), -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat((p, q), -1))
    rest = x[..., 2 * r:]
    return torch.cat((join(a, b), rest), -1), torch.cat((join(size, size), rest.abs()), -1)


def check(got, ref, size, d, extra=16):
    tol = (d / 2 + 8 + extra) * U * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol + 1e-37).all()), f"off by {(err / (tol + 1e-37)).max():.3g} of the bound"


def _qk(**kw):
    far = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 9)]
    a = dict(qo=far[0], ld_qo=64, ko=far[1], ld_ko=64, out_dt=1, q=far[2], ld_q=64, k=far[3], ld_k=64, in_dt=1, qw=None,
             kw=None, freq=far[4], rot=8, pos=None, eps=1e-6, flags=0, B=1, T=4, Hq=4, Hk=4, d=16)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.load().mamba_qk_norm_rotary(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(qo=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(ko=None), -1), (dict(freq=None), -1),
    (dict(in_dt=3), -1), (dict(out_dt=-1), -1), (dict(rot=7), -1), (dict(rot=18), -1), (dict(rot=-2), -1),
    (dict(flags=4), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(ld_q=63), -1), (dict(ld_ko=63), -1),
    (dict(B=-1), -1), (dict(Hq=-1), -1), (dict(d=0), -2), (dict(d=257), -2), (dict(T=1 << 60), -1),
    (dict(qo=FAKE, ko=FAKE), -1), (dict(qo=FAKE, k=FAKE), -1), (dict(qo=FAKE, q=ctypes.c_void_p(0x100002)), -1),
])
def test_qk_norm_refusals(kw, code):
    assert _qk(**kw) == code
    assert m.mamba_last_error()


def test_qk_norm_in_place_and_empty_calls_pass_the_host_checks():
    for kw in (dict(qo=FAKE, q=FAKE), dict(Hk=0, k=None, ko=None)):
        assert _qk(**kw) != 0 and "overlap" not in m.mamba_last_error()  # refused for the device alone here
    assert _qk(B=0) == 0 and _qk(T=0) == 0 and _qk(Hq=0, Hk=0) == 0


def _hn(**kw):
    far = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 9)]
    a = dict(out=far[0], ld_out=64, out_dt=1, y=far[1], ld_y=64, z=far[2], ld_z=64, in_dt=1, w=None, eps=1e-5, rows=4,
             H=4, d=16)
    a.update(kw)
    return m.load().mamba_head_norm_gated(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(out=None), dict(y=None), dict(ld_out=63), dict(ld_y=63), dict(ld_z=63), dict(eps=2.0),
                                dict(in_dt=9), dict(rows=-1), dict(H=-1), dict(rows=1 << 60), dict(out=FAKE, z=FAKE)])
def test_head_norm_refusals(kw):
    assert _hn(**kw) == -1


def test_python_refusals():
    q = torch.zeros(2, 3, 4, 16)
    for kw in (dict(positions=torch.zeros(2, 3)), dict(positions=torch.zeros(2, 2, dtype=torch.int64)),
               dict(inv_freq=torch.zeros(2, 2)), dict(q_weight=torch.ones(15)), dict(inv_freq=torch.zeros(2).double())):
        with pytest.raises(ValueError):
            m.mamba_qk_norm_rotary(q.clone(), None, q, None, **kw)
    with pytest.raises(ValueError):
        m.mamba_qk_norm_rotary(q.clone(), None, q, q)
    with pytest.raises(ValueError):
        m.mamba_qk_norm_rotary(q.clone()[..., :8], None, q, None)
    with pytest.raises(ValueError):
        m.mamba_head_norm_gated(q.clone(), q, q[:1])
    with pytest.raises(ValueError):
        m.mamba_head_norm_gated(q.clone(), q, None, torch.ones(8))


# ------------------------------------------------------------------ on the GPU

def inputs(seed, B, T, Hq, Hk, d, rot, dtype, far=True):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(B, T, h, d, generator=g).to(DT[dtype]).cuda() for h in (Hq, Hk))
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    freq = (10000.0 ** (-torch.arange(0, rot, 2).float() / max(rot, 1))).cuda() if rot else None
    pos = torch.randint(0, 1 << 20 if far else T, (B, T), generator=g).cuda()
    return q, k, qw, kw, freq, pos


@pytest.mark.gpu
@pytest.mark.parametrize("din,dout", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 64), (128, 128), (128, 0), (256, 32), (96, 48), (80, 80), (72, 8),
                                   (17, 6), (1, 0), (2, 2), (250, 100)])
@pytest.mark.parametrize("interleaved,l2", [(False, True), (True, False)])
def test_qk_norm(cuda_lib, d, rot, interleaved, l2, din, dout):
    q, k, qw, kw, freq, pos = inputs(d + rot, 2, 5, 3, 2, d, rot, din)
    if l2:
        qw = None
    qo, ko = (torch.full(t.shape, float("nan"), dtype=DT[dout], device="cuda") for t in (q, k))
    m.mamba_qk_norm_rotary(qo, ko, q, k, qw, kw, freq, pos, l2=l2, interleaved=interleaved)
    torch.cuda.synchronize()
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        check(got, *ref_turn(ref_norm(x, w, 1e-6, l2), freq, pos, interleaved), d)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (1, 1, 16, 0), (128, 1, 16, 16), (1, 700, 5, 1), (3, 333, 2, 7),
                                       (4, 1500, 12, 4)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_norm_shapes(cuda_lib, B, T, Hq, Hk, interleaved):
    q, k, qw, kw, freq, _ = inputs(B + T, B, T, Hq, max(Hk, 1), 128, 64, "bf16")
    k, ko = (k, torch.empty_like(k)) if Hk else (None, None)
    qo = torch.empty_like(q)
    m.mamba_qk_norm_rotary(qo, ko, q, k, qw, kw, freq, None, interleaved=interleaved)
    torch.cuda.synchronize()
    pos = torch.arange(T).expand(B, T)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        if x is not None:
            check(got, *ref_turn(ref_norm(x, w, 1e-6, False), freq, pos, interleaved), 128)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions_and_any_frequency(cuda_lib, interleaved):
    """The angle is exact to 2^-32 turns beside the 2^-53 of a turn per position of its table entry."""
    q = torch.randn(1, 8, 2, 64, generator=torch.Generator().manual_seed(1)).cuda()
    freq = torch.tensor([1.0, 0.1, 1e-4, 1e-7, 0.0, -0.5, 3.0, 7.5] * 4).cuda()
    pos = torch.tensor([[0, 1, -1, 1 << 20, (1 << 31) + 7, -(1 << 25), 12345678, 99]]).cuda()
    out = torch.empty_like(q)
    m.mamba_qk_norm_rotary(out, None, q, None, None, None, freq, pos, interleaved=interleaved)
    ref, size = ref_turn(ref_norm(q, None, 1e-6, False), freq, pos, interleaved)
    # both sides' angles: 2^-53 relative in the reference's product and in the table, at most 7.5 * 2^31 radians
    check(out, ref, size, 64, 16 + 2 * 7.5 * 2 ** 31 * 2 ** -53 / U)


@pytest.mark.gpu
@pytest.mark.parametrize("d,pad", [(128, 8), (64, 3), (40, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qk_norm_in_place_on_packed_columns(cuda_lib, d, pad, dtype):
    q, k, qw, kw, freq, pos = inputs(3, 2, 9, 3, 2, d, 32, dtype)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    m.mamba_qk_norm_rotary(qo, ko, q, k, qw, kw, freq, pos)
    buf = torch.full((2, 9, 5 * d + 3 * pad), 7.0, dtype=DT[dtype], device="cuda")
    pq = buf[..., pad:pad + 3 * d].unflatten(-1, (3, d))
    pk = buf[..., 2 * pad + 3 * d:2 * pad + 5 * d].unflatten(-1, (2, d))
    pq.copy_(q)
    pk.copy_(k)
    m.mamba_qk_norm_rotary(pq, pk, pq, pk, qw, kw, freq, pos)
    torch.cuda.synchronize()
    tol = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -20  # another reduction order: a value may round the other way
    assert float((pq.float() - qo.float()).abs().max()) <= tol * float(qo.float().abs().max())
    assert float((pk.float() - ko.float()).abs().max()) <= tol * float(ko.float().abs().max())
    for lo, hi in ((0, pad), (pad + 3 * d, 2 * pad + 3 * d), (2 * pad + 5 * d, 3 * pad + 5 * d)):
        assert bool((buf[..., lo:hi] == 7).all())


@pytest.mark.gpu
def test_norms_of_zero_and_extreme_rows(cuda_lib):
    q = torch.randn(1, 6, 2, 64, generator=torch.Generator().manual_seed(2)).cuda()
    q[0, 0] = 0
    q[0, 1] *= 1e-15
    q[0, 2] *= 1e15
    q[0, 3, 0, 5] = float("inf")
    q[0, 4, 1, 5] = float("nan")
    out = torch.empty_like(q)
    m.mamba_qk_norm_rotary(out, None, q, None, l2=True)
    ref = ref_norm(q, None, 1e-6, True)
    rows = [(0, 0), (0, 1), (1, 0), (1, 1), (2, 0), (2, 1), (3, 1), (4, 0), (5, 0), (5, 1)]
    for t, h in rows:  # a row does not see its neighbours
        check(out[0, t, h], ref[0, t, h], ref[0, t, h].abs(), 64)
    assert not bool(torch.isfinite(out[0, 3, 0, 5])) and bool(torch.isnan(out[0, 4, 1]).all())
    z = torch.full_like(q, -200.0)
    z[0, :, 1] = 200.0
    m.mamba_head_norm_gated(out, q, z)
    assert not out[0, 0].any() and not out[0, 1, 0].any() and not out[0, 5, 0].any()
    check(out[0, 5, 1], 200 * ref_norm(q, None, 1e-5, False)[0, 5, 1],
          200 * ref_norm(q, None, 1e-5, False)[0, 5, 1].abs(), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("din,dout", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,T,H,d", [(1, 1, 1, 64), (128, 1, 24, 64), (2, 333, 5, 128), (3, 7, 4, 256), (2, 5, 3, 96),
                                     (2, 5, 3, 33), (1, 2, 2, 600), (1, 3000, 6, 128)])
def test_head_norm(cuda_lib, B, T, H, d, din, dout):
    g = torch.Generator().manual_seed(d)
    y, z = (torch.randn(B, T, H, d, generator=g).to(DT[din]).cuda() for _ in range(2))
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    for zz, ww in ((z, w), (None, w), (z, None)):
        out = torch.full(y.shape, float("nan"), dtype=DT[dout], device="cuda")
        m.mamba_head_norm_gated(out, y, zz, ww)
        ref = ref_norm(y, ww, 1e-5, False)
        if zz is not None:
            zd = zz.cpu().double()
            ref = ref * zd * torch.sigmoid(zd)
        check(out, ref, ref.abs(), d)
    if din == dout:  # in place
        want = out
        m.mamba_head_norm_gated(y, y, z)
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_head_norms_in_a_graph_on_another_stream(cuda_lib):
    q, k, qw, kw, freq, pos = inputs(3, 4, 1, 8, 4, 128, 64, "bf16")
    qo, ko, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)

    def call():
        m.mamba_qk_norm_rotary(qo, ko, q, k, qw, kw, freq, pos)
        m.mamba_head_norm_gated(out, qo, q, qw)

    call()
    want = [t.clone() for t in (qo, ko, out)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for t in (qo, ko, out):
            t.zero_()
        call()
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((qo, ko, out), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for t in (qo, ko, out):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((qo, ko, out), want))
