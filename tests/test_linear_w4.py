"""Projections with 4-bit weights against their sum in 64 bits.

A product of a bf16 and a difference q - z of at most 8 bits is exact in 32 bits.  The
sum of K of them, the scales' products and the residual take at most K + 64 additions
and products, each off by at most 2^-23 (a tensor core may cut instead of round) of a
partial sum, which is at most the sum of the terms' sizes.  A bf16 result adds half a
step, 2^-8 of the value.
"""
import ctypes

import pytest
import torch

import selective_state_space_conv1d_gb300 as m

FAKE = ctypes.c_void_p(0x100000)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def weights(seed, N, K, group, scales="bf16", zeros=False, junk=True):
    """Random 4-bit weights: (q, scales, zeros or None) on the CPU, what lies past K random too."""
    g = torch.Generator().manual_seed(seed)
    G = -(-K // group)
    q = torch.randint(0, 256, (N, -(-K // 32) * 16), generator=g, dtype=torch.uint8)
    if not junk:
        v = values(q, K)
        v = torch.nn.functional.pad(v, (0, q.shape[1] * 2 - K))
        q = (v[:, 0::2] | v[:, 1::2] << 4).to(torch.uint8)
    s = (torch.rand(N, G, generator=g) + 0.5).to(DT[scales]) * K ** -0.5
    z = torch.randint(0, 16, (N, G), generator=g, dtype=torch.uint8) if zeros else None
    return q, s.to(DT[scales]), z


def values(q, K):
    return torch.stack((q & 15, q >> 4), -1).flatten(1)[:, :K]


def reference(a, q, s, z, group, residual=None):
    """(C, the sum of the terms' sizes) in 64 bits."""
    K = a.shape[1]
    spread = lambda t: t.double().repeat_interleave(group, 1)[:, :K]  # noqa: E731
    w = (values(q, K).double() - (8 if z is None else spread(z))) * spread(s)
    a = a.cpu().double()
    c, size = a @ w.T, a.abs() @ w.abs().T
    if residual is not None:
        c, size = c + residual.cpu().double(), size + residual.cpu().double().abs()
    return c, size


def check(got, ref, size, K):
    tol = (K + 64) * 2.0 ** -23 * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol + 1e-37).all()), f"off by {(err / (tol + 1e-37)).max():.3g} of the bound"


# ------------------------------------------------------------------ refusals, on the CPU

def _call(**kw):
    far = [ctypes.c_void_p(0x10000000 * i) for i in range(1, 9)]
    a = dict(c=far[0], ld_c=64, c_dt=0, a=far[1], ld_a=96, q=far[2], ld_q=48, s=far[3], ld_s=1, s_dt=1, z=far[4], ld_z=1,
             group=128, r=None, ld_r=0, M=4, N=64, K=96)
    assert set(kw) <= set(a)
    a.update(kw)
    return m.load().mamba_linear_w4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), -1), (dict(a=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(c_dt=2), -1),
    (dict(s_dt=-1), -1), (dict(ld_c=63), -1), (dict(ld_a=95), -1), (dict(ld_q=47), -1), (dict(ld_q=56), -1),
    (dict(ld_a=100), -1), (dict(K=97), -1), (dict(group=32), -1), (dict(group=32, ld_s=3), -1), (dict(group=16), -2),
    (dict(group=0), -2), (dict(group=-128), -2), (dict(M=-1), -1), (dict(N=-1), -1), (dict(K=0), -1), (dict(M=1 << 31), -1), (dict(K=(1 << 30) + 1), -1), (dict(N=(1 << 30) + 1), -1),
    (dict(a=ctypes.c_void_p(0x20000008)), -1), (dict(q=ctypes.c_void_p(0x30000008)), -1), (dict(c=FAKE, a=FAKE), -1),
    (dict(c=FAKE, q=FAKE), -1), (dict(c=FAKE, s=FAKE), -1), (dict(c=FAKE, z=FAKE), -1), (dict(r=FAKE, ld_r=63), -1),
    (dict(c=FAKE, r=FAKE, ld_r=64, c_dt=1), -1), (dict(c=FAKE, r=FAKE, ld_r=65), -1),
    (dict(s=ctypes.c_void_p(0x40000001)), -1),
])
def test_refusals(kw, code):
    assert _call(**kw) == code
    assert m.mamba_last_error()


def test_empty_calls_and_an_update_in_place_pass_the_host_checks():
    assert _call(M=0) == 0 and _call(N=0) == 0
    assert _call(c=FAKE, r=FAKE, ld_r=64) != 0 and "overlap" not in m.mamba_last_error()  # refused for the device alone


def test_python_refusals():
    q, s, z = weights(0, 16, 96, 32, zeros=True)
    a, c = torch.zeros(2, 96, dtype=torch.bfloat16), torch.zeros(2, 16)
    bad = [dict(q=q.int()), dict(q=q[:, :32]), dict(q=q[0]), dict(scales=s[:, :2]), dict(scales=s.double()),
           dict(zeros=z.int()), dict(zeros=z[:8]), dict(a=a.float()), dict(a=a[0]), dict(c=c[:1]), dict(c=c.half()),
           dict(residual=c.bfloat16()), dict(group=64), dict(group=0), dict(residual=c[:, :8])]
    for kw in bad:
        args = dict(c=c, a=a, q=q, scales=s, zeros=z, residual=None, group=32)
        args.update(kw)
        group = args.pop("group")
        with pytest.raises((ValueError, TypeError)):
            m.mamba_linear_w4(*args.values(), group=group)


# ------------------------------------------------------------------ on the GPU

def run(a, q, s, z, group, out="f32", residual=None):
    M, N = a.shape[0], q.shape[0]
    c = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
    m.mamba_linear_w4(c, a, *(None if t is None else t.cuda() for t in (q, s, z)), residual, group=group)
    return c


def activations(seed, M, K):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(M, -(-K // 8) * 8, generator=g).to(torch.bfloat16)
    return wide.cuda()[:, :K]


ROWS = [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 515]


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", ROWS)
def test_rows(cuda_lib, M, group):
    N, K = 272, 416
    q, s, z = weights(M, N, K, group, "bf16" if M % 2 else "f32", M % 3 != 0)
    a = activations(M, M, K)
    check(run(a, q, s, z, group), *reference(a, q, s, z, group), K)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8, 40, 150])
@pytest.mark.parametrize("N,K", [(1, 1), (1, 4096), (3, 8), (16, 31), (17, 33), (127, 127), (128, 128), (129, 129),
                                 (130, 1000), (1003, 1000), (300, 48), (48, 5120), (2560, 160), (33, 257), (5000, 64)])
def test_sizes(cuda_lib, M, N, K):
    for group, scales, zeros, out in ((32, "f32", True, "bf16"), (128, "bf16", False, "f32")):
        q, s, z = weights(N + K, N, K, group, scales, zeros)
        a = activations(M, M, K)
        check(run(a, q, s, z, group, out), *reference(a, q, s, z, group), K)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 64, 300])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("scales,zeros", [("f32", False), ("f32", True), ("bf16", False), ("bf16", True)])
def test_types_and_residual(cuda_lib, M, out, scales, zeros):
    N, K = 520, 640
    q, s, z = weights(7, N, K, 64, scales, zeros)
    a = activations(3, M, K)
    r = torch.randn(M, N, generator=torch.Generator().manual_seed(5)).cuda()
    check(run(a, q, s, z, 64, out, r), *reference(a, q, s, z, 64, r), K)
    if out == "f32":  # in place
        want = run(a, q, s, z, 64, out, r)
        m.mamba_linear_w4(r, a, q.cuda(), s.cuda(), None if z is None else z.cuda(), r, group=64)
        assert torch.equal(r, want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8, 12, 130])
def test_strided_views_and_what_is_around_them(cuda_lib, M):
    N, K, group = 130, 200, 32
    q, s, z = weights(1, N, K, group, "bf16", True)
    a = activations(1, M, K)
    want = run(a, q, s, z, group)
    wide_a = torch.full((M, 264), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_a[:, 16:16 + K] = a
    wide_q = torch.randint(0, 256, (N, 160), dtype=torch.uint8, device="cuda")
    wide_q[:, 16:16 + q.shape[1]] = q.cuda()
    wide_s = torch.full((N, 11), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_s[:, 3:3 + s.shape[1]] = s.cuda()
    wide_z = torch.full((N, 9), 99, dtype=torch.uint8, device="cuda")
    wide_z[:, 1:1 + s.shape[1]] = z.cuda()
    for pad in (1, 4):
        wide_c = torch.full((M + 2, N + 2 * pad), 7.0, device="cuda")
        c = wide_c[1:M + 1, pad:pad + N]
        m.mamba_linear_w4(c, wide_a[:, 16:16 + K], wide_q[:, 16:16 + q.shape[1]], wide_s[:, 3:3 + s.shape[1]],
                          wide_z[:, 1:1 + s.shape[1]], group=group)
        assert torch.equal(c, want)
        wide_c[1:M + 1, pad:pad + N] = 7.0
        assert bool((wide_c == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8, 70, 260])
def test_what_lies_past_k_is_ignored(cuda_lib, M):
    K, N = 77, 200
    q, s, z = weights(2, N, K, 32, zeros=True)
    clean, _, _ = weights(2, N, K, 32, zeros=True, junk=False)
    wide = torch.full((M, 80), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = activations(2, M, K)
    a = wide[:, :K]
    got = run(a, q, s, z, 32)
    check(got, *reference(a, q, s, z, 32), K)
    assert torch.equal(got, run(a, clean, s, z, 32))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 20, 140])
def test_a_row_keeps_to_itself(cuda_lib, M):
    N, K = 144, 512
    q, s, z = weights(4, N, K, 128)
    a = activations(4, M, K)
    want = run(a, q, s, z, 128)
    a[1, 100] = float("nan")
    a[2, 5] = float("inf")
    got = run(a, q, s, z, 128)
    rows = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(got[rows], want[rows])
    assert bool(got[1].isnan().all()) and not bool(got[2].isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 16, 128])
def test_extreme_weights(cuda_lib, M):
    N, K, group = 64, 256, 64
    a = activations(5, M, K)
    for fill, zero in ((0x00, 0), (0xff, 0), (0x00, 127), (0xff, 15), (0x80, 8)):
        q = torch.full((N, K // 2), fill, dtype=torch.uint8)
        z = torch.full((N, K // group), zero, dtype=torch.uint8)
        for scale in (0.0, -1.5, 2.0 ** 100, 2.0 ** -100):
            s = torch.full((N, K // group), scale)
            check(run(a, q, s, z, group), *reference(a, q, s, z, group), K)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 2560, 5120), (4, 50000, 2560), (24, 10240, 2560), (128, 10240, 2560),
                                   (700, 5120, 2560), (4100, 1100, 1536)])
def test_large(cuda_lib, M, N, K):
    q, s, z = weights(6, N, K, 128, "bf16", True)
    a = activations(6, M, K)
    got = run(a, q, s, z, 128)
    rows = torch.arange(0, N, max(1, N // 97))
    pick = torch.arange(0, M, max(1, M // 61))
    check(got[pick][:, rows], *reference(a[pick], q[rows], s[rows], z[rows], 128), K)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,scales,zeros,out", [(20480, 2560, "bf16", True, "f32"), (20003, 2603, "f32", False, "bf16"),
                                                  (60001, 1000, "bf16", False, "f32"), (1300, 32768 + 40, "f32", True, "f32"),
                                                  (10001, 9000, "bf16", True, "bf16")])
def test_one_row_of_many_weights(cuda_lib, N, K, scales, zeros, out):
    q, s, z = weights(9, N, K, 128, scales, zeros)
    a = activations(9, 1, K)
    r = torch.randn(1, N, generator=torch.Generator().manual_seed(5)).cuda()
    got = run(a, q, s, z, 128, out, r)
    rows = torch.cat((torch.arange(0, N, max(1, N // 97)), torch.arange(N - 17, N)))
    pick = lambda t: None if t is None else t[rows]  # noqa: E731
    check(got[:, rows], *reference(a, q[rows], s[rows], pick(z), 128, r[:, rows]), K)
    assert bool(got.isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 6, 50, 300])
def test_repeats_on_other_streams_and_in_a_graph(cuda_lib, M):
    N, K, group = 1040, 1536, 128
    q, s, z = (t.cuda() for t in weights(8, N, K, group, "bf16", True))
    a = activations(8, M, K)
    c = torch.empty(M, N, device="cuda")

    def call():
        m.mamba_linear_w4(c, a, q, s, z, group=group)

    call()
    want = c.clone()
    st = torch.cuda.Stream()
    for _ in range(3):
        c.zero_()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            call()
        st.synchronize()
        assert torch.equal(c, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        c.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)
    assert m.mamba_device_faults() == 0
