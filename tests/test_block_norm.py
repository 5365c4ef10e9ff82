"""The residual stream between two blocks against its formula in 64 bits.

Tolerances in units of U = 2^-24.  A sum of D squares goes through at most D / 128 + 60
additions (a thread's own, its warp's, the warps'); the root, the quotient and the
products with weights add 8 more.  So n is off by (D / 128 + 68) U |n|, the gate, the
scale and the sum make that (D / 128 + 72) U |scale gate n| + U |x'|, and out moves by
its own part of x' and by the length of all of it.  A bf16 output adds half a step,
2^-8 of the value.
"""
import ctypes

import pytest
import torch

import selective_state_space_conv1d_gb300 as m

FAKE = ctypes.c_void_p(0x100000)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def reference(x, y, pre, post, gate, scale, eps=1e-5):
    """((x', its bound), (out, its bound)) in 64 bits; gate broadcasts to x."""
    x, y = x.cpu().double(), y.cpu().double()
    D = x.shape[-1]
    chain = D / 128 + 72
    n = y
    if post is not None:
        n = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * post.cpu().double()
    if gate is not None:
        n = n * gate.cpu().double()
    s = x + scale * n
    tol = chain * U * (scale * n).abs() + U * s.abs()
    if pre is None:
        return (s, tol), None
    rms = torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    w = pre.cpu().double()
    out = s / rms * w
    moved = tol.square().mean(-1, keepdim=True).sqrt() / rms
    return (s, tol), (out, tol / rms * w.abs() + out.abs() * (moved + chain * U))


def check(got, ref_tol):
    ref, tol = ref_tol
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol + 1e-37).all()), f"off by {(err / (tol + 1e-37)).max():.3g} of the bound"


# ------------------------------------------------------------------ refusals, on the CPU

def _call(**kw):
    far = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 9)]
    a = dict(xo=far[0], ld_xo=64, out=far[1], ld_o=64, o_dt=1, x=far[2], ld_x=64, y=far[3], ld_y=64, y_dt=1, pre=far[4],
             post=far[5], gate=far[6], ld_g=64, g_dt=0, g_rows=1, scale=1.0, eps=1e-5, M=4, D=64)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.load().mamba_block_norm(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(xo=None), dict(x=None), dict(y=None), dict(out=None), dict(pre=None), dict(o_dt=2), dict(y_dt=-1), dict(g_dt=5),
    dict(ld_xo=63), dict(ld_o=63), dict(ld_x=63), dict(ld_y=63), dict(ld_g=63), dict(g_rows=-1), dict(M=-1), dict(D=0),
    dict(eps=-1.0), dict(eps=2.0), dict(eps=float("nan")), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(M=1 << 40, D=1 << 20), dict(xo=FAKE, x=FAKE, ld_x=72), dict(xo=FAKE, y=FAKE), dict(out=FAKE, y=FAKE),
    dict(out=FAKE, x=FAKE), dict(xo=FAKE, out=FAKE), dict(xo=FAKE, gate=FAKE), dict(out=FAKE, pre=FAKE),
    dict(xo=FAKE, post=FAKE), dict(x=ctypes.c_void_p(0x3000002)),
])
def test_refusals(kw):
    assert _call(**kw) == -1
    assert m.mamba_last_error()


def test_empty_calls_and_an_update_in_place_pass_the_host_checks():
    assert _call(M=0) == 0
    for kw in (dict(xo=FAKE, x=FAKE), dict(out=None, pre=None), dict(gate=None), dict(post=None)):
        assert _call(**kw) != 0 and "overlap" not in m.mamba_last_error() and "NULL" not in m.mamba_last_error()


def test_python_refusals():
    x, y, w = torch.zeros(2, 3, 16), torch.zeros(2, 3, 16, dtype=torch.bfloat16), torch.ones(16)
    good = dict(x_out=x.clone(), out=y.clone(), x=x, y=y, pre_weight=w, post_weight=w, gate=None)
    for kw in (dict(x=x.bfloat16()), dict(x_out=x.bfloat16()), dict(x_out=x[:1]), dict(y=y[:, :2]), dict(y=y.half()),
               dict(out=y.half()), dict(out=y[..., :8]), dict(pre_weight=w[:8]), dict(post_weight=w.bfloat16()),
               dict(gate=w[:8]), dict(gate=torch.ones(3, 16)), dict(gate=torch.ones(2, 3, 8)), dict(gate=w.half()),
               dict(x=x[0, 0]), dict(gate=torch.ones(1, 2, 3, 16))):
        with pytest.raises((ValueError, TypeError)):
            m.mamba_block_norm(*{**good, **kw}.values())


# ------------------------------------------------------------------ on the GPU

def inputs(seed, shape, y="bf16", gate=None, gate_dtype="f32"):
    g = torch.Generator().manual_seed(seed)
    D = shape[-1]
    x, yy = 2 * torch.randn(*shape, generator=g), torch.randn(*shape, generator=g).to(DT[y])
    pre, post = 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(D, generator=g)
    gs = dict(none=None, channel=(D,), sequence=(shape[0], D), token=shape)[gate or "none"]
    gg = torch.randn(*gs, generator=g).to(DT[gate_dtype]).cuda() if gs else None
    return x.cuda(), yy.cuda(), pre.cuda(), post.cuda(), gg


def spread(gate, shape):
    if gate is None or gate.dim() in (1, len(shape)):
        return gate
    return gate[:, None]


def run(x, y, pre, post, gate, scale, out="bf16", **kw):
    xo = torch.full_like(x, float("nan"))
    o = torch.full(x.shape, float("nan"), dtype=DT[out], device="cuda")
    m.mamba_block_norm(xo, o, x, y, pre, post, gate, scale=scale, **kw)
    return xo, o


LENGTHS = [1, 7, 8, 64, 96, 100, 768, 1000, 1024, 1032, 2560, 4096, 5120, 8192, 8200, 9001, 16384, 16392, 20000]


@pytest.mark.gpu
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("D", LENGTHS)
def test_lengths(cuda_lib, D, post):
    x, y, pre, post_w, gate = inputs(D, (2, 3, D), gate="channel")
    post_w = post_w if post else None
    got = run(x, y, pre, post_w, gate, 0.5)
    for g, r in zip(got, reference(x, y, pre, post_w, gate, 0.5)):
        check(g, r)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["none", "channel", "sequence", "token"])
@pytest.mark.parametrize("gate_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("y,out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("D", [640, 333])
def test_types_and_gates(cuda_lib, gate, gate_dtype, y, out, D):
    shape = (3, 5, D)
    x, yy, pre, post, gg = inputs(3, shape, y, gate, gate_dtype)
    got = run(x, yy, pre, post, gg, -1.25, out)
    for g, r in zip(got, reference(x, yy, pre, post, spread(gg, shape), -1.25)):
        check(g, r)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 128, 700])
@pytest.mark.parametrize("D", [768, 2560])
def test_rows(cuda_lib, M, D):
    for gate in ("none", "token"):
        x, y, pre, post, gg = inputs(M, (M, D), gate=gate, gate_dtype="bf16")
        for g, r in zip(run(x, y, pre, post, gg, 0.75), reference(x, y, pre, post, gg, 0.75)):
            check(g, r)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [512, 257])
def test_in_place_and_without_the_next_norm(cuda_lib, D):
    x, y, pre, post, gate = inputs(4, (2, 7, D), gate="sequence")
    want, out = run(x, y, pre, post, gate, 2.0)
    only = torch.empty_like(x)
    m.mamba_block_norm(only, None, x, y, None, post, gate, scale=2.0)
    assert torch.equal(only, want)
    o = torch.empty_like(out)
    m.mamba_block_norm(x, o, x, y, pre, post, gate, scale=2.0)
    assert torch.equal(x, want) and torch.equal(o, out)


@pytest.mark.gpu
def test_a_plain_sum_and_norm_is_rmsnorm_of_the_sum(cuda_lib):
    """Without a gate, a scale or a norm after the block: mamba_rmsnorm of x + y."""
    x, y, pre, _, _ = inputs(5, (6, 1536))
    xo, out = run(x, y, pre, None, None, 1.0)
    assert torch.equal(xo, x + y.float())
    ref = torch.empty_like(out)
    m.mamba_rmsnorm(ref, xo, pre)
    assert float((ref.float() - out.float()).abs().max()) <= 2.0 ** -7 * float(ref.float().abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("D,pad", [(256, 8), (256, 3), (100, 1)])
def test_strided_views_and_what_is_around_them(cuda_lib, D, pad):
    B, T = 2, 5
    x, y, pre, post, gate = inputs(6, (B, T, D), gate="token")
    want = run(x, y, pre, post, gate, 0.5)
    wide = {}
    for name, t in (("xo", x), ("out", y), ("x", x), ("y", y), ("gate", gate)):
        w = torch.full((B, T, D + 2 * pad), 7.0, dtype=t.dtype, device="cuda")
        w[..., pad:pad + D] = t
        wide[name] = w
    v = {n: w[..., pad:pad + D] for n, w in wide.items()}
    m.mamba_block_norm(v["xo"], v["out"], v["x"], v["y"], pre, post, v["gate"], scale=0.5)
    # another order of the sums where the views are not aligned
    for got, ref in zip((v["xo"], v["out"]), reference(x, y, pre, post, gate, 0.5)):
        check(got, ref)
    if pad % 8 == 0:
        assert torch.equal(v["xo"], want[0]) and torch.equal(v["out"], want[1])
    for w in wide.values():
        w[..., pad:pad + D] = 7.0
        assert bool((w == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [640, 333])
def test_zeros_extremes_and_rows_apart(cuda_lib, D):
    x, y, pre, post, _ = inputs(7, (6, D), "f32")
    x[0] = 0
    y[0] = 0
    y[1] *= 1e-15
    y[2] *= 1e15
    x[2] *= 1e15
    y[3, 5] = float("nan")
    x[4, 5] = float("inf")
    xo, out = run(x, y, pre, post, None, 1.0, "f32")
    assert not xo[0].any() and not out[0].any()
    rows = [0, 1, 2, 5]
    for g, r in zip((xo, out), reference(x[rows], y[rows], pre, post, None, 1.0)):
        check(g[rows], r)
    assert bool(out[3].isnan().all()) and bool(out[4, 5].isnan())


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph(cuda_lib):
    x, y, pre, post, gate = inputs(8, (4, 9, 768), gate="sequence")
    xo, out = torch.empty_like(x), torch.empty_like(y)

    def call():
        m.mamba_block_norm(xo, out, x, y, pre, post, gate, scale=0.5)

    call()
    want = xo.clone(), out.clone()
    st = torch.cuda.Stream()
    xo.zero_(), out.zero_()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    st.synchronize()
    assert torch.equal(xo, want[0]) and torch.equal(out, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    xo.zero_(), out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(xo, want[0]) and torch.equal(out, want[1])
