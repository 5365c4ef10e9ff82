"""The example block: a prompt and decoded tokens against one longer prompt, and
against the block's formulas in 64 bits."""
import importlib.util
import os

import pytest
import torch

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_delta_block.py")
_spec = importlib.util.spec_from_file_location("gated_delta_block", _PATH)
block = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(block)


def _rounded(x):
    return x.to(torch.bfloat16).double()


def _plain(s, layers, hidden):
    """The blocks over [B, T, d_model] from zero states, 64 bits between the stored
    bf16 activations."""
    x = hidden.double()
    B, T, _ = x.shape
    for w in layers:
        w = {k: v.double() for k, v in w.items()}
        h = _rounded(x / (x.square().mean(-1, keepdim=True) + block.EPS).sqrt() * w["norm"])
        p = _rounded(h @ w["w_in"].T)
        qkv = torch.cat([torch.zeros(B, s.taps - 1, s.conv, dtype=x.dtype), p[..., :s.conv]], 1)
        u = w["conv_b"] + sum(qkv[:, i:i + T] * w["conv_w"][:, i] for i in range(s.taps))
        u = _rounded(u * torch.sigmoid(u))
        q, k, v = u.split([s.keys, s.keys, s.values], -1)
        angle = torch.arange(T, dtype=x.dtype)[:, None] * w["inv_freq"]
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]

        def turned(t):
            t = t.reshape(B, T, s.k_heads, s.d)
            t = t / (t.square().sum(-1, keepdim=True) + block.EPS).sqrt()
            lo, hi, rest = t.split([s.rot // 2, s.rot // 2, s.d - s.rot], -1)
            t = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, rest], -1)
            return _rounded(t).repeat_interleave(s.v_heads // s.k_heads, 2)

        q, k, v = turned(q), turned(k), v.reshape(B, T, s.v_heads, s.d)
        z, a, b = p[..., s.conv:].split([s.values, s.v_heads, s.v_heads], -1)
        alpha = torch.exp(-w["A_log"].exp() * torch.nn.functional.softplus(a + w["dt_bias"]))
        beta = torch.sigmoid(b)
        S = torch.zeros(B, s.v_heads, s.d, s.d, dtype=x.dtype)
        y = torch.empty(B, T, s.v_heads, s.d, dtype=x.dtype)
        for t in range(T):
            S = S * alpha[:, t, :, None, None]
            e = beta[:, t, :, None] * (v[:, t] - (S @ k[:, t, :, :, None])[..., 0])
            S = S + e[..., None] * k[:, t, :, None, :]
            y[:, t] = (S @ q[:, t, :, :, None])[..., 0] * s.d ** -0.5
        y = _rounded(y)
        z = z.reshape(B, T, s.v_heads, s.d)
        y = y / (y.square().mean(-1, keepdim=True) + block.EPS).sqrt() * w["out_norm"] * z * torch.sigmoid(z)
        x = x + _rounded(y).reshape(B, T, s.values) @ w["w_out"].T
    return x


# A block rounds six tensors to bf16.  Where two evaluations differ before a rounding
# the rounded values differ by a step at most, 2^-7 of a value, so by 2^-8 in the mean
# over a tensor at the very worst; the update's relative error is then below
# 6 * 2^-8 per block, of which the second block sees the first's as well.
N_LAYERS = 2
TOL = N_LAYERS * 6 * 2.0 ** -8


def _close(got, want, start):
    got, want, start = (t.double().cpu() for t in (got, want, start))
    err = (got - want).norm() / (want - start).norm()
    assert err < TOL, f"relative error of the blocks' update {err:.2e}, allowed {TOL:.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("prompt, tokens", [(70, 6), (1, 3), (130, 1)])
def test_prompt_and_decoded_tokens(prompt, tokens):
    s = block.Sizes(d_model=256, k_heads=2, v_heads=4, d=64, rot=32)
    g = torch.Generator(device="cuda").manual_seed(prompt)
    layers = [block.random_weights(s, g) for _ in range(N_LAYERS)]
    B, T = 3, prompt + tokens
    x = torch.randn(B, T, s.d_model, generator=g, device="cuda")

    whole, whole_states = x.clone(), block.States(s, N_LAYERS, B)
    block.prefill(s, layers, whole, whole_states)
    _close(whole, _plain(s, [{k: v.cpu() for k, v in w.items()} for w in layers], x.cpu()), x)

    states = block.States(s, N_LAYERS, B)
    first = x[:, :prompt].contiguous()
    block.prefill(s, layers, first, states)
    _close(first, whole[:, :prompt], x[:, :prompt])
    decode = block.Decode(s, layers, states)
    for t in range(prompt, T):
        decode.hidden.copy_(x[:, t])
        decode.launch()
        _close(decode.hidden, whole[:, t], x[:, t])
    assert states.position.flatten().tolist() == [T] * B
    err = (states.delta - whole_states.delta).norm() / whole_states.delta.norm()
    assert err < TOL
    assert block.m.mamba_device_faults() == 0
