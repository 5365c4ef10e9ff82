"""The gated delta rule (prefill and step) against its recurrence in 64 bits.

Tolerance of the f32 arithmetic: a value that is a chain of products over dk
key components and up to two chunks of 64 tokens, each term off by at most
2^-22 of its size (an f32 rounding, or an operand held as two 11-bit halves),
is off by at most (dk + 128 + 16) 2^-22 of its largest term; keys of at most
unit length make the rule a contraction, so earlier errors do not grow.  The
reference returns the largest terms (|S| over all tokens, and scale |S| |q|).
A bf16 y adds half a step, 2^-8 of the value.
"""
import ctypes
import math

import pytest
import torch

import selective_state_space_conv1d_gb300 as m

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: the calls below fail before any device work
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ reference

def make(seed, B, T, Hk, Hv, dk, dv, dtype="f32", state=True, corr=0.5, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(r(B, T, Hk, dk) + corr * r(Hk, dk)), k=unit(r(B, T, Hk, dk) + corr * r(Hk, dk)),
             v=r(B, T, Hv, dv), a=0.5 * r(B, T, Hv), b=r(B, T, Hv))
    x = {n: t.to(DT[dtype]) for n, t in x.items()}
    x["A_log"] = torch.log(1 + 15 * torch.rand(Hv, generator=g))
    x["dt_bias"] = torch.log(torch.expm1(torch.exp(math.log(1e-3) + torch.rand(Hv, generator=g) * math.log(100))))
    x["state_in"] = 0.3 * r(B, Hv, dv, dk) if state else None
    return {n: t.to(device) if t is not None else None for n, t in x.items()}


def reference(x, scale=None):
    """(y, S, largest terms of y, largest |S|) in 64 bits, the latter [B, Hv, 1, 1]."""
    q, k, v, a, b = (x[n].detach().cpu().double() for n in ("q", "k", "v", "a", "b"))
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    q, k = (t.repeat_interleave(Hv // Hk, 2) for t in (q, k))
    bias = x["dt_bias"].cpu().double() if x["dt_bias"] is not None else 0.0
    alpha = torch.exp(-torch.exp(x["A_log"].cpu().double()) * torch.nn.functional.softplus(a + bias, threshold=1000))
    beta = torch.sigmoid(b)
    S = x["state_in"].detach().cpu().double().clone() if x["state_in"] is not None else \
        torch.zeros(B, Hv, dv, dk, dtype=torch.float64)
    scale = dk ** -0.5 if scale is None else scale
    y = torch.zeros(B, T, Hv, dv, dtype=torch.float64)
    ms = S.abs().amax((2, 3), keepdim=True)
    my = torch.zeros(B, Hv, dtype=torch.float64)
    for t in range(T):
        S = S * alpha[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S @ k[:, t, :, :, None])[..., 0])
        S = S + u[..., None] * k[:, t, :, None]
        y[:, t] = scale * (S @ q[:, t, :, :, None])[..., 0]
        ms = torch.maximum(ms, S.abs().amax((2, 3), keepdim=True))
        my = torch.maximum(my, abs(scale) * (S.abs() @ q[:, t, :, :, None].abs())[..., 0].amax(-1))
    return y, S, my, ms


def run_prefill(x, scale=None, y_dtype=None, inplace=False):
    y = torch.empty(x["v"].shape, dtype=y_dtype or x["v"].dtype, device="cuda").fill_(float("nan"))
    B, _, Hv, dv = x["v"].shape
    s_in = x["state_in"].clone() if x["state_in"] is not None else None
    s_out = s_in if inplace else torch.full((B, Hv, dv, x["q"].shape[3]), float("nan"), device="cuda")
    m.mamba_gated_delta_prefill(y, x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"], s_in, s_out,
                                scale=scale)
    torch.cuda.synchronize()
    if s_in is not None and not inplace:
        assert torch.equal(s_in, x["state_in"])
    return y, s_out


def check(x, y, s, scale=None, what=""):
    ry, rs, my, ms = reference(x, scale)
    dk = x["q"].shape[3]
    eps = (dk + 144) * 2.0 ** -22
    tol = eps * my[:, None, :, None] + (2.0 ** -8 * ry.abs() if y.dtype == torch.bfloat16 else 0)
    ey = (y.cpu().double() - ry).abs()
    assert bool((ey <= tol).all()), f"{what} y off by {(ey / tol.clamp(min=1e-300)).max():.3g} of the bound"
    if s is not None:
        es = (s.cpu().double() - rs).abs()
        assert bool((es <= eps * ms).all()), f"{what} state off by {(es / (eps * ms)).max():.3g} of the bound"


# ------------------------------------------------------------------ host checks

def _prefill(**kw):
    a = dict(y=FAKE, ld_y=64, y_dt=1, q=FAKE, ld_q=64, k=FAKE, ld_k=64, v=FAKE, ld_v=64, a=FAKE, ld_a=4, b=FAKE, ld_b=4,
             in_dt=1, A=FAKE, bias=None, scale=1.0, s_in=None, s_out=None, B=1, T=4, Hk=4, Hv=4, dk=16, dv=16, ws=None,
             ws_bytes=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.load().mamba_gated_delta_prefill(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(a=None), -1),
    (dict(b=None), -1), (dict(A=None), -1), (dict(y_dt=2), -1), (dict(in_dt=-1), -1),
    (dict(ld_y=63), -1), (dict(ld_q=63), -1), (dict(ld_k=63), -1), (dict(ld_v=63), -1), (dict(ld_a=3), -1),
    (dict(ld_b=3), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(Hk=0), -1), (dict(Hv=0), -1), (dict(Hv=6), -1),
    (dict(dk=0), -2), (dict(dk=257), -2), (dict(dv=0), -2), (dict(dv=1025), -2),
    (dict(T=1 << 62), -1), (dict(B=1 << 45, T=1 << 45), -1), (dict(ws_bytes=-1), -1),
    (dict(), -1),  # every tensor at one address: y overlaps q
    (dict(y=ctypes.c_void_p(0x900001)), -1),  # a bf16 tensor at an odd address
])
def test_prefill_refusals(kw, code):
    assert _prefill(**kw) == code
    assert m.mamba_last_error()


def test_prefill_overlap_refusals():
    far = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 10)]
    ok = dict(y=far[0], q=far[1], k=far[2], v=far[3], a=far[4], b=far[5], A=far[6])
    state = 4 * 4 * 16 * 16
    for kw in (dict(s_out=far[1]), dict(s_out=far[0]), dict(s_out=ctypes.c_void_p(far[7].value + state // 2), s_in=far[7]),
               dict(ws=far[3], ws_bytes=64), dict(ws=far[0], ws_bytes=64)):
        assert _prefill(**{**ok, **kw}) == -1 and "overlaps" in m.mamba_last_error()
    # columns of one packed buffer do not overlap: refused for the device only
    row = 4 * 16
    packed = {n: ctypes.c_void_p(0x1000000 + 2 * row * i) for i, n in enumerate(("q", "k", "v", "y"))}
    rc = _prefill(**{**ok, **packed}, ld_q=4 * row, ld_k=4 * row, ld_v=4 * row, ld_y=4 * row)
    assert rc != 0 and "overlaps" not in m.mamba_last_error()
    packed["y"] = ctypes.c_void_p(packed["y"].value - 2)
    rc = _prefill(**{**ok, **packed}, ld_q=4 * row, ld_k=4 * row, ld_v=4 * row, ld_y=4 * row)
    assert rc == -1 and "overlaps" in m.mamba_last_error()


def test_empty_batch_is_ok():
    assert _prefill(B=0) == 0


def _step(**kw):
    a = dict(y=FAKE, ld_y=64, y_dt=1, q=FAKE, ld_q=64, k=FAKE, ld_k=64, v=FAKE, ld_v=64, a=FAKE, ld_a=4, b=FAKE, ld_b=4,
             in_dt=1, A=FAKE, bias=None, scale=1.0, state=FAKE, layer=0, n_layers=1, B=1, Hk=4, Hv=4, dk=16, dv=16)
    a.update(kw)
    return m.load().mamba_gated_delta_step_batched(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), -1), (dict(layer=1), -1), (dict(n_layers=0), -1), (dict(state=None), -1), (dict(q=None), -1),
    (dict(ld_y=63), -1), (dict(B=-1), -1), (dict(Hv=6), -1), (dict(dk=300), -2), (dict(), -1),
])
def test_step_refusals(kw, code):
    assert _step(**kw) == code


def test_python_refusals():
    x = make(0, 2, 5, 2, 4, 16, 8)
    args = lambda **kw: [{**x, **kw}[n] for n in ("q", "k", "v", "a", "b", "A_log", "dt_bias")]  # noqa: E731
    y, s = torch.empty_like(x["v"]), torch.zeros(2, 4, 8, 16)
    bad = [dict(k=x["k"][:, :, :1]), dict(k=x["k"].double()), dict(a=x["a"][:, :, :3]), dict(b=x["b"].to(torch.bfloat16)),
           dict(A_log=x["A_log"].double()), dict(dt_bias=x["dt_bias"][:3]), dict(v=x["v"].transpose(2, 3)),
           dict(q=x["q"].transpose(0, 1))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            m.mamba_gated_delta_prefill(y, *args(**kw), None, s)
    with pytest.raises(ValueError):
        m.mamba_gated_delta_prefill(y[:, :4], *args(), None, s)
    with pytest.raises(ValueError):
        m.mamba_gated_delta_prefill(y, *args(), s[:1], s)
    with pytest.raises(ValueError):
        m.mamba_gated_delta_prefill(y, *args(), None, s.transpose(2, 3))


def test_reference_is_the_delta_rule():
    """One unit key: S k becomes v exactly at beta = 1, and alpha = 1 keeps the rest."""
    x = make(1, 1, 1, 1, 1, 8, 4)
    x["a"].fill_(-1e4)
    x["b"].fill_(1e4)
    x["q"] = x["k"].clone()
    y, S, _, _ = reference(x, 1.0)
    assert torch.allclose(y[0, 0, 0], x["v"][0, 0, 0].double(), atol=1e-6)
    p = torch.eye(8, dtype=torch.float64) - torch.outer(*[x["k"][0, 0, 0].double()] * 2)
    assert torch.allclose(S[0, 0] @ p, x["state_in"][0, 0].double() @ p, atol=1e-6)


# ------------------------------------------------------------------ on the GPU

LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 331]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", LENGTHS)
def test_prefill_lengths(cuda_lib, T, dtype):
    x = make(T, 2, T, 2, 4, 128, 128, dtype, state=T % 2 == 1, device="cuda")
    y, s = run_prefill(x)
    check(x, y, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hk,Hv,dk,dv", [
    (1, 1, 64, 64), (2, 2, 64, 128), (1, 3, 128, 64), (1, 1, 128, 256), (2, 4, 96, 128), (3, 3, 72, 40), (1, 2, 17, 5),
    (1, 1, 1, 1), (1, 1, 256, 128), (1, 2, 200, 33), (2, 2, 8, 8), (1, 1, 130, 24), (1, 1, 64, 1000), (2, 6, 126, 126),
])
@pytest.mark.parametrize("T", [3, 150])
def test_prefill_heads(cuda_lib, Hk, Hv, dk, dv, T, dtype):
    x = make(7 * dk + dv, 2, T, Hk, Hv, dk, dv, dtype, device="cuda")
    y, s = run_prefill(x)
    check(x, y, s)


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["keep", "drop", "drop_some", "beta0", "beta1", "same_key", "huge_v", "tiny_v", "mixed_v",
                                  "small_k", "zero_k", "fast", "no_bias", "scale"])
@pytest.mark.parametrize("dtype,T", [("bf16", 150), ("f32", 150), ("bf16", 5)])
def test_prefill_extremes(cuda_lib, case, dtype, T):
    x = make(11, 1, T, 2, 2, 128, 64, dtype, device="cuda")
    scale = None
    if case == "keep":
        x["a"].fill_(-float("inf"))       # alpha = 1
    elif case == "drop":
        x["a"].fill_(float("inf"))        # alpha = 0: every token starts anew
    elif case == "drop_some":
        x["a"][:, 5::37] = float("inf")
        x["a"][:, 3::29] = 1e4
    elif case == "beta0":
        x["b"].fill_(-float("inf"))
    elif case == "beta1":
        x["b"].fill_(float("inf"))
        x["a"].fill_(-20.0)
    elif case == "same_key":              # the triangular system at its worst
        x["k"][:] = x["k"][:, :1]
        x["b"].fill_(float("inf"))
        x["a"].fill_(-30.0)
    elif case == "huge_v":
        x["v"] *= 1e8
    elif case == "tiny_v":
        x["v"] *= 1e-12
        x["state_in"] *= 1e-12
    elif case == "mixed_v":               # magnitudes jump from token to token and component to component
        x["v"][:, 70:] *= 1e6
        x["v"][:, 100:] *= 1e-9
        x["v"][..., ::3] *= 1e-5
    elif case == "small_k":
        x["k"] *= 1e-3
        x["q"] *= 1e3
    elif case == "zero_k":
        x["k"][:, ::2] = 0
        x["q"][:, 1::3] = 0
    elif case == "fast":                  # decays of e^-20 a token beside slow ones
        x["A_log"].fill_(math.log(20.0))
        x["a"][:, ::2] = 1.0
        x["a"][:, 1::2] = -15.0
    elif case == "no_bias":
        x["dt_bias"] = None
    elif case == "scale":
        scale = -3.0
    y, s = run_prefill(x, scale)
    if case == "mixed_v":  # a bound by the largest value of each value component, not of the head
        for n in range(3):
            xs = dict(x, v=x["v"][..., n::3], state_in=x["state_in"][:, :, n::3])
            check(xs, y[..., n::3], s[:, :, n::3], scale, case)
    else:
        check(x, y, s, scale, case)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 100])
def test_non_finite_values_stay_in_their_components(cuda_lib, T):
    x = make(5, 1, T, 1, 1, 64, 64, "bf16", device="cuda")
    clean_y, clean_s = run_prefill(x)
    x["v"][0, T // 2, 0, 3] = float("inf")
    x["v"][0, 0, 0, 9] = float("nan")
    y, s = run_prefill(x)
    others = [n for n in range(64) if n not in (3, 9)]
    assert torch.equal(y[..., others], clean_y[..., others]) and torch.equal(s[:, :, others], clean_s[:, :, others])
    assert bool(torch.isnan(y[0, :, 0, 9]).all())
    assert bool((~torch.isfinite(s[0, 0, [3, 9]])).all())
    if T // 2 > 64:
        assert torch.equal(y[:, :64, :, 3], clean_y[:, :64, :, 3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T1,T2", [(1, 1), (64, 64), (100, 77), (5, 200)])
def test_prefill_continues(cuda_lib, T1, T2, dtype):
    x = make(3, 2, T1 + T2, 1, 2, 64, 64, dtype, device="cuda")
    part = lambda lo, hi, s: {n: t[:, lo:hi].contiguous() if n in ("q", "k", "v", "a", "b") else t  # noqa: E731
                              for n, t in dict(x, state_in=s).items()}
    y1, s1 = run_prefill(part(0, T1, x["state_in"]))
    y2, s2 = run_prefill(part(T1, T1 + T2, s1), inplace=True)
    check(x, torch.cat((y1, y2), 1), s2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_packed_columns(cuda_lib, T, pad, dtype):
    """q, k, v, a, b and y as columns of wider rows, the columns between them NaN."""
    x = make(9, 3, T, 2, 4, 64, 64, dtype, device="cuda")
    y0, s0 = run_prefill(x)
    cols, at = {}, pad
    for n, w in (("q", 128), ("k", 128), ("v", 256), ("a", 4), ("b", 4)):
        cols[n] = (at, w)
        at += w + pad
    buf = torch.full((3, T, at + (-at) % 8), float("nan"), dtype=DT[dtype], device="cuda")
    px = dict(x)
    for n, (c, w) in cols.items():
        view = buf[..., c:c + w]
        px[n] = view.unflatten(-1, x[n].shape[2:]) if n in ("q", "k", "v") else view
        px[n].copy_(x[n])
    ybuf = torch.full((3, T, 256 + 2 * pad), 5.0, dtype=DT[dtype], device="cuda")
    y = ybuf[..., pad:pad + 256].unflatten(-1, (4, 64))
    s = torch.empty_like(s0)
    m.mamba_gated_delta_prefill(y, px["q"], px["k"], px["v"], px["a"], px["b"], x["A_log"], x["dt_bias"],
                                x["state_in"], s)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(s, s0)
    assert bool((ybuf[..., :pad] == 5).all()) and bool((ybuf[..., pad + 256:] == 5).all())


@pytest.mark.gpu
def test_prefill_states_optional_and_y_types(cuda_lib):
    x = make(4, 2, 90, 2, 2, 64, 64, "bf16", state=False, device="cuda")
    y, s = run_prefill(x)
    check(x, y, s)
    y32, s32 = run_prefill(x, y_dtype=torch.float32)
    check(x, y32, s32)
    assert torch.equal(y32.to(torch.bfloat16), y) and torch.equal(s, s32)
    yn = torch.empty_like(y)
    m.mamba_gated_delta_prefill(yn, x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"], None, None)
    assert torch.equal(yn, y)
    # no tokens: the state passes through
    e = {n: (t[:, :0] if n in ("q", "k", "v", "a", "b") else t) for n, t in x.items()}
    so = torch.full_like(s, 3.0)
    m.mamba_gated_delta_prefill(y[:, :0], e["q"], e["k"], e["v"], e["a"], e["b"], e["A_log"], e["dt_bias"], s, so)
    assert torch.equal(so, s)
    m.mamba_gated_delta_prefill(y[:, :0], e["q"], e["k"], e["v"], e["a"], e["b"], e["A_log"], e["dt_bias"], None, so)
    assert not so.any()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,Hv,dk,dv,dtype", [(1, 2, 2, 64, 64, "bf16"), (5, 2, 6, 128, 128, "bf16"),
                                                  (3, 1, 1, 96, 40, "f32"), (2, 1, 2, 17, 130, "f32"),
                                                  (33, 3, 3, 256, 8, "bf16")])
def test_steps(cuda_lib, B, Hk, Hv, dk, dv, dtype):
    """Steps on a middle layer's slab follow the recurrence; the other slabs stay; a step is a T = 1 prefill."""
    T, L = 5, 3
    x = make(21, B, T, Hk, Hv, dk, dv, dtype, device="cuda")
    state = torch.randn(L, B, Hv, dv, dk, device="cuda")
    state[1] = x["state_in"]
    keep = state.clone()
    y = torch.empty_like(x["v"])
    for t in range(T):
        one = {n: x[n][:, t] for n in ("q", "k", "v", "a", "b")}
        pre = {n: x[n][:, t:t + 1].contiguous() for n in ("q", "k", "v", "a", "b")}
        yp, sp = run_prefill(dict(x, **pre, state_in=state[1].clone()))
        m.mamba_gated_delta_step_batched(y[:, t], one["q"], one["k"], one["v"], one["a"], one["b"], x["A_log"],
                                         x["dt_bias"], state, 1)
        torch.cuda.synchronize()
        assert torch.equal(yp[:, 0], y[:, t]) and torch.equal(sp, state[1])
    check(x, y, state[1])
    assert torch.equal(state[0], keep[0]) and torch.equal(state[2], keep[2])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 130])
def test_streams_graphs_and_repeats(cuda_lib, T):
    """The call runs on the current stream, is captured into a graph, and repeats bit for bit."""
    x = make(31, 2, T, 2, 4, 128, 128, "bf16", device="cuda")
    y0, s0 = run_prefill(x)
    y1, s1 = run_prefill(x)
    assert torch.equal(y0, y1) and torch.equal(s0, s1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y, s = torch.zeros_like(y0), torch.zeros_like(s0)
    call = lambda: m.mamba_gated_delta_prefill(y, x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"],  # noqa: E731
                                               x["dt_bias"], x["state_in"], s)
    with torch.cuda.stream(st):
        call()
    st.synchronize()
    assert torch.equal(y, y0) and torch.equal(s, s0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    y.zero_()
    s.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(s, s0)
    assert m.mamba_device_faults() == 0


@pytest.mark.gpu
def test_batch_rows_are_independent(cuda_lib):
    x = make(41, 5, 140, 1, 2, 64, 128, "bf16", device="cuda")
    y, s = run_prefill(x)
    one = {n: t[3:4].contiguous() if n not in ("A_log", "dt_bias") else t for n, t in x.items()}
    y3, s3 = run_prefill(one)
    check(one, y3, s3)
    tol = (64 + 144) * 2.0 ** -22
    assert float((s3[0] - s[3]).abs().max()) <= 2 * tol * float(s[3].abs().max() + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,Hv,T,dk,dv", [(1, 1, 1, 3000, 128, 128), (1, 2, 4, 1500, 64, 64), (2, 1, 3, 1100, 128, 256)])
def test_long_prefills_of_few_heads(cuda_lib, B, Hk, Hv, T, dk, dv):
    x = make(51, B, T, Hk, Hv, dk, dv, "bf16", device="cuda")
    x["dt_bias"] -= 4  # slow decays: the first tokens still count at the end
    y, s = run_prefill(x)
    check(x, y, s)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,Hv,T,dk,dv,dtype,y32", [
    (2, 90, 90, 200, 64, 64, "bf16", False), (3, 26, 52, 330, 128, 136, "bf16", False), (1, 200, 200, 70, 128, 64, "bf16", True),
    (2, 79, 79, 140, 64, 64, "f32", False), (4, 60, 60, 65, 40, 8, "bf16", False),
])
def test_more_items_than_sms(cuda_lib, B, Hk, Hv, T, dk, dv, dtype, y32):
    """Items that begin on one SM and end on the next; and the same without scratch, one item a CTA."""
    x = make(61, B, T, Hk, Hv, dk, dv, dtype, device="cuda")
    x["dt_bias"] -= 3
    y, s = run_prefill(x, y_dtype=torch.float32 if y32 else None)
    check(x, y, s)
    y2, s2 = torch.empty_like(y), torch.empty_like(s)
    m.mamba_gated_delta_prefill(y2, x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"], x["state_in"], s2,
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2)  # the state is handed over in full
    assert m.mamba_device_faults() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,Hv,T,dk,dv,dtype,state", [
    (1, 2, 2, 2048, 128, 128, "bf16", True), (1, 1, 3, 1990, 64, 128, "bf16", False), (1, 2, 4, 1200, 96, 200, "bf16", True),
    (2, 3, 3, 1111, 64, 64, "f32", True), (1, 1, 1, 1025, 128, 40, "f32", False), (1, 8, 16, 3000, 128, 128, "bf16", True),
])
def test_sequences_cut_into_parts(cuda_lib, B, Hk, Hv, T, dk, dv, dtype, state):
    x = make(71, B, T, Hk, Hv, dk, dv, dtype, state=state, device="cuda")
    x["dt_bias"] -= 4
    assert m.mamba_gated_delta_workspace_bytes(B, T, Hk, Hv, dk, dv, 1 if dtype == "bf16" else 0) > 0
    y, s = run_prefill(x)
    check(x, y, s)
    y1, s1 = run_prefill(x)
    assert torch.equal(y, y1) and torch.equal(s, s1)
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")  # too little: one pass over the sequence
    m.mamba_gated_delta_prefill(y1, x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"], x["state_in"], s1,
                                workspace=ws)
    torch.cuda.synchronize()
    check(x, y1, s1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T", [("bf16", 2048), ("f32", 1999)])
def test_parts_with_the_state_in_place(cuda_lib, dtype, T):
    # the first part still needs the state when the last one may have written it
    x = make(72, 1, T, 4, 8, 64, 128, dtype, state=True, device="cuda")
    assert m.mamba_gated_delta_workspace_bytes(1, T, 4, 8, 64, 128, 1 if dtype == "bf16" else 0) > 0
    y, s = run_prefill(x)
    for _ in range(5):
        state, y1 = x["state_in"].clone(), torch.empty_like(y)
        m.mamba_gated_delta_prefill(y1, x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"], state, state)
        assert torch.equal(y, y1) and torch.equal(s, state)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "a", "b"])
@pytest.mark.parametrize("t", [37, 64, 130])
def test_nan_stays_in_its_head_and_group(cuda_lib, dtype, name, t):
    x = make(73, 2, 200, 2, 4, 64, 64, dtype, state=True, device="cuda")
    y, s = run_prefill(x)
    x[name][1, t, 1] = float("nan")
    y1, s1 = run_prefill(x)
    heads = [2, 3] if name in ("q", "k") else [1]  # of the second sequence
    others = [h for h in range(4) if h not in heads]
    assert torch.equal(y[0], y1[0]) and torch.equal(s[0], s1[0])
    assert torch.equal(y[1, :, others], y1[1, :, others]) and torch.equal(s[1, others], s1[1, others])
    assert torch.equal(y[1, :t // 16 * 16], y1[1, :t // 16 * 16])
    assert y1[1, t, heads].isnan().all()
    if name != "q":
        assert y1[1, t:, heads].isnan().all() and s1[1, heads].isnan().all()
