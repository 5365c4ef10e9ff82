"""Blocks with 4-bit projections: the block call against its sequence of calls, bit for
bit, its decode graph, its refusals, the weights' helpers; and a token's whole path --
blocks, the sum and norm after them, a 4-bit head, log probabilities -- against 64 bits.

The projections' own accuracy is tested in test_linear_w4, the mixer's in test_layer_gpu.
"""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_conv1d_gb300 as m
from oracle import layer as OL
from selective_state_space_conv1d_gb300 import _binding, synth

PROJ = ("in_proj_w", "x_proj_w", "dt_proj_w", "out_proj_w")


# ------------------------------------------------------------------ the weights, on the CPU

@pytest.mark.parametrize("K", [1, 31, 32, 77, 160])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_and_pack(K, group, zeros):
    """A value is off by at most half a step of its group, and by a step where the rounded
    scale clips the group's end: a bf16 scale is off by 2^-8 of itself, times 15 values."""
    g = torch.Generator().manual_seed(K + group)
    w = torch.randn(5, K, generator=g)
    for dt in (torch.float32, torch.bfloat16):
        q = m.quantize_w4(w, group, zeros=zeros, scale_dtype=dt)
        assert q.q.shape == (5, -(-K // 32) * 16) and q.scales.shape == (5, -(-K // group)) and q.scales.dtype == dt
        step = q.scales.float().repeat_interleave(group, 1)[:, :K]
        slack = 0.5 + (0.5 if zeros else 0) + 15 * 2.0 ** -8  # a zero point rounds by half a step
        assert bool(((m.dequantize_w4(q, K) - w).abs() <= slack * step).all())
        v = m.unpack_w4(q.q, K)
        assert torch.equal(m.pack_w4(v), q.q) and int(v.max()) <= 15
    assert torch.equal(m.dequantize_w4(m.quantize_w4(torch.zeros(2, K), group, zeros=zeros), K), torch.zeros(2, K))


def test_packing_is_low_half_first():
    v = torch.arange(16).repeat(3)[None, :40]
    q = m.pack_w4(v)
    assert q.shape == (1, 32) and q[0, :3].tolist() == [0x10, 0x32, 0x54] and not q[0, 20:].any()


def test_helpers_refuse():
    w = torch.randn(3, 40)
    for bad in (lambda: m.quantize_w4(w, 16), lambda: m.quantize_w4(w[0]), lambda: m.quantize_w4(w.int()),
                lambda: m.quantize_w4(w, scale_dtype=torch.float16), lambda: m.pack_w4(w),
                lambda: m.pack_w4(torch.full((2, 2), 16)), lambda: m.pack_w4(torch.full((2, 2), -1))):
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------------ refusals, on the CPU

def block_weights(seed, dm=64, Di=128, N=16, K=4, R=8, group=32, zeros=False, four=PROJ, device="cpu"):
    """(weights for the calls, the oracle's f64 weights) with the projections `four` in 4 bits."""
    p = synth.layer_params(seed, dm, Di, N, K, R, parity=True)
    w, ref = {}, dict(p)
    for k, v in p.items():
        t = None if v is None else torch.from_numpy(np.ascontiguousarray(v, np.float32))
        if k in four:
            q = m.quantize_w4(t, group, zeros=zeros)
            ref[k] = m.dequantize_w4(q, t.shape[1]).double().numpy()
            t = m.W4(*(x.to(device) if isinstance(x, torch.Tensor) else x for x in q))
        elif t is not None:
            t = (t.to(torch.bfloat16) if k.endswith("proj_w") else t).to(device)
        w[k] = t
    return w, ref


@pytest.mark.parametrize("change,code", [
    (dict(group=48), -2), (dict(group=0), -2), (dict(scale_dtype=3), -1), (dict(scales=None), -1), (dict(ld_q=16), -1),
    (dict(ld_q=40), -1), (dict(ld_s=1), -1), (dict(q=0x100008), -1), (dict(scales=0x100001), -1),
])
def test_block_refuses_before_any_launch(change, code):
    w, _ = block_weights(1)
    s = m.layer_struct(w)
    assert isinstance(s, _binding._MambaLayerW4)
    for k, v in change.items():
        setattr(s.in_proj, k, v)
    hidden, ws = torch.zeros(2, 64), torch.zeros(1 << 16, dtype=torch.uint8)
    rc = m.load().mamba_layer_w4_prefill(hidden.data_ptr(), ctypes.byref(s), None, None, None, None, 1, 2, ws.data_ptr(),
                                         ws.numel(), None)
    assert rc == code and m.mamba_last_error()


def test_block_refuses_a_missing_weight_and_null():
    lib = m.load()
    s = m.layer_struct(block_weights(1)[0])
    s.out_proj.q = None  # and no bf16 weight either
    hidden = torch.zeros(2, 64)
    assert lib.mamba_layer_w4_prefill(hidden.data_ptr(), ctypes.byref(s), None, None, None, None, 1, 2, hidden.data_ptr(),
                                      1 << 20, None) == -1
    assert lib.mamba_layer_w4_prefill(hidden.data_ptr(), None, None, None, None, None, 1, 2, None, 0, None) == -1
    assert lib.mamba_layer_w4_step(hidden.data_ptr(), None, None, None, 0, 1, 1, None, 0, None) == -1
    h = ctypes.c_void_p()
    assert lib.mamba_layer_w4_decode_graph_create(ctypes.byref(h), None, 1, None, None, None, 1, None, 0) == -1
    assert "mamba_layer_w4_decode_graph_create" in m.mamba_last_error() and not h.value


def test_python_refuses_shapes():
    w, _ = block_weights(1)
    for k in PROJ:
        for bad in (w[k]._replace(q=w[k].q[:-1]), w[k]._replace(group=64 if k != "dt_proj_w" else 0),
                    w[k]._replace(scales=w[k].scales.double()), w[k]._replace(zeros=w[k].scales)):
            with pytest.raises((ValueError, TypeError)):
                m.layer_struct({**w, k: bad})


# ------------------------------------------------------------------ on the GPU

def linear(c, a, w, residual=None):
    if isinstance(w, m.W4):
        m.mamba_linear_w4(c, a, w.q, w.scales, w.zeros, residual, group=w.group)
    else:
        m.mamba_linear_bf16(c, a, w, residual)


def block_by_calls(hidden, w, conv_state, ssm_state):
    """hidden [B, T, dm] and the states in place, by the block's documented calls."""
    B, T, dm = hidden.shape
    Di, N = w["A_log"].shape
    rows = w["x_proj_w"].q.shape[0] if isinstance(w["x_proj_w"], m.W4) else w["x_proj_w"].shape[0]
    R = rows - 2 * N
    new = lambda c: torch.empty(B * T, c, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x2 = hidden.view(B * T, dm)
    h, xz, u, xd, dt, y = new(dm), new(2 * Di), new(Di), new((rows + 7) // 8 * 8)[:, :rows], new(Di), new(Di)
    m.mamba_rmsnorm(h, x2, w["norm_w"])
    linear(xz, h, w["in_proj_w"])
    v = lambda t: t.view(B, T, -1) if t.is_contiguous() else t.unflatten(0, (B, T))  # noqa: E731
    x3, z3 = v(xz)[..., :Di], v(xz)[..., Di:]
    m.mamba_conv1d_silu_prefill(v(u), x3, w["conv_w"], w["conv_b"], conv_state, conv_state)
    linear(xd, u, w["x_proj_w"])
    linear(dt, xd[:, :R], w["dt_proj_w"])
    m.mamba_selective_scan_prefill(v(y), v(u), v(dt), v(xd)[..., R:R + N], v(xd)[..., R + N:R + 2 * N], w["A_log"],
                                   w["D"], w["dt_bias"], z3, ssm_state, ssm_state)
    linear(x2, y, w["out_proj_w"], x2)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (1, 40), (2, 150), (130, 1)])
@pytest.mark.parametrize("four,group,zeros", [(PROJ, 32, True), (PROJ, 128, False), (("in_proj_w", "out_proj_w"), 64, False)])
def test_block_is_its_calls(cuda_lib, B, T, four, group, zeros):
    w, _ = block_weights(B + T, four=four, group=group, zeros=zeros, device="cuda")
    g = torch.Generator().manual_seed(B * T)
    hidden = torch.randn(B, T, 64, generator=g).cuda()
    conv, ssm = torch.randn(B, 128, 4, generator=g).cuda(), torch.randn(B, 128, 16, generator=g).cuda()
    want = [t.clone() for t in (hidden, conv, ssm)]
    block_by_calls(want[0], w, want[1], want[2])
    m.mamba_layer_prefill(hidden, w, conv, conv, ssm, ssm)
    assert all(torch.equal(a, b) for a, b in zip((hidden, conv, ssm), want))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 8, 40])
def test_step_is_a_prefill_of_one_and_the_graph_is_its_steps(cuda_lib, B):
    L, dm, Di = 3, 64, 128
    layers = [block_weights(l, four=PROJ if l != 1 else (), device="cuda")[0] for l in range(L)]  # one bf16 block between
    g = torch.Generator().manual_seed(B)
    h0 = torch.randn(B, dm, generator=g).cuda()
    conv0, ssm0 = torch.randn(L, B, Di, 4, generator=g).cuda(), torch.randn(L, B, Di, 16, generator=g).cuda()
    h1, conv1, ssm1 = h0.clone(), conv0.clone(), ssm0.clone()
    h2, conv2, ssm2 = h0.clone(), conv0.clone(), ssm0.clone()
    for l in range(L):
        m.mamba_layer_step(h1, layers[l], conv1, ssm1, l)
        m.mamba_layer_prefill(h2.view(B, 1, dm), layers[l], conv2[l], conv2[l], ssm2[l], ssm2[l])
    assert torch.equal(h1, h2) and torch.equal(conv1, conv2) and torch.equal(ssm1, ssm2)
    h3, conv3, ssm3 = h0.clone(), conv0.clone(), ssm0.clone()
    with m.LayerDecodeGraph(layers, h3, conv3, ssm3) as graph:
        graph.launch()
        torch.cuda.synchronize()
        assert torch.equal(h3, h1) and torch.equal(conv3, conv1) and torch.equal(ssm3, ssm1)
        for l in range(L):  # a second token continues
            m.mamba_layer_step(h1, layers[l], conv1, ssm1, l)
        graph.launch()
        torch.cuda.synchronize()
    assert torch.equal(h3, h1) and torch.equal(ssm3, ssm1)
    assert m.mamba_device_faults() == 0


def _bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(1, 33), (2, 9)])
def test_a_tokens_whole_path(cuda_lib, B, T):
    """A prompt through two 4-bit blocks, a 4-bit gated branch beside the second, the sum with
    its gate and the last norm, the 4-bit head, and what its logits say; then the same in a
    graph.  The reference stores what the calls store in bf16; a rounding that falls the other
    way there is a step of 2^-8 that spreads over a row's 64 values, so the stream may be off by
    a few hundredths of the blocks' update (as test_layer_gpu's), the logits by that share of
    their size."""
    dm, V = 64, 501
    g = torch.Generator().manual_seed(5)
    blocks = [block_weights(10 + i, device="cuda") for i in range(2)]
    head = m.quantize_w4(torch.randn(V, dm, generator=g) * 0.3, 64, zeros=True)
    branch = m.quantize_w4(torch.randn(dm, dm, generator=g) * dm ** -0.5, 32)
    post, pre = 1 + 0.1 * torch.randn(dm, generator=g), 1 + 0.1 * torch.randn(dm, generator=g)
    gate = torch.rand(B, dm, generator=g)
    x0 = torch.randn(B, T, dm, generator=g)
    tokens = torch.randint(0, V, (B * T,), generator=g)
    dev = lambda q: m.W4(*(t.cuda() if isinstance(t, torch.Tensor) else t for t in q))  # noqa: E731
    head_d, branch_d, post_d, pre_d, gate_d = dev(head), dev(branch), post.cuda(), pre.cuda(), gate.cuda()
    hidden = x0.cuda()
    y, out = (torch.empty(B, T, dm, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    n = torch.empty(B * T, dm, device="cuda", dtype=torch.bfloat16)
    logits = torch.empty(B * T, V, device="cuda")
    lp, h = torch.empty(B * T, device="cuda"), torch.empty(B * T, device="cuda")
    tl, ti = torch.empty(B * T, 4, device="cuda"), torch.empty(B * T, 4, device="cuda", dtype=torch.int64)
    t_d = tokens.cuda()

    def run():
        for w, _ in blocks:
            m.mamba_layer_prefill(hidden, w)
        m.mamba_rmsnorm(n, hidden.view(B * T, dm), pre_d)
        linear(y.view(B * T, dm), n, branch_d)
        m.mamba_block_norm(hidden, out, hidden, y, pre_d, post_d, gate_d, scale=0.5)
        linear(logits, out.view(B * T, dm), head_d)
        m.mamba_token_logprobs(lp, h, tl, ti, logits, t_d)

    run()
    # the reference
    x = x0.double().numpy().reshape(B * T, dm)
    start = x
    for _, p in blocks:
        x = OL.layer_prefill(x, p, B, T, store=_bf16)[0]
    yr = _bf16(_bf16(OL.rmsnorm(x, pre.numpy())) @ m.dequantize_w4(branch, dm).double().numpy().T)
    x = x + 0.5 * gate.double().numpy().repeat(T, 0) * OL.rmsnorm(yr, post.numpy())
    update = np.sqrt(np.mean((x - start) ** 2))
    assert np.abs(hidden.double().cpu().numpy().reshape(B * T, dm) - x).max() <= 0.08 * update
    lr = _bf16(OL.rmsnorm(x, pre.numpy())) @ m.dequantize_w4(head, dm).double().numpy().T
    assert np.abs(logits.double().cpu().numpy() - lr).max() <= 0.08 * np.sqrt(np.mean(lr ** 2)) * 4
    # what is said of the logits as they are
    ld = logits.double()
    ref = torch.log_softmax(ld, -1)
    bound = (V / 256 + 110) * 2.0 ** -24 + 4 * 2.0 ** -24 * (10 + ref.abs())
    assert bool(((lp.double() - ref[torch.arange(B * T), t_d]).abs() <= bound[torch.arange(B * T), t_d]).all())
    assert float((h.double() + (ref.exp() * ref).sum(-1)).abs().max()) <= float(20 * bound.max())
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(ti, order)
    # captured
    outs = (hidden, out, logits, lp, h, tl, ti)
    want = [t.clone() for t in outs]
    hidden.copy_(x0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t in outs:
        t.zero_()
    hidden.copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert m.mamba_device_faults() == 0
