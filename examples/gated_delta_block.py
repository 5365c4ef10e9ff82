"""A recurrent block on the gated delta rule: prompt and graph-captured decode.

    hidden += W_out . gated_norm(delta_rule(norm_turn(silu(conv(q k v)))))

from this library's calls: RMSNorm, the bf16 projections, the causal conv with
SiLU, the norms of queries and keys with the position rotation, the gated delta
rule, the output norm with its SiLU(z) gate.  A prompt goes through prefill();
decode() records one token through all blocks as a CUDA graph, whose launches
then advance the blocks' states and positions.

    python examples/gated_delta_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_conv1d_gb300 as m  # noqa: E402

EPS = 1e-6


class Sizes:
    """Model width, key heads, value heads, head size, conv taps, turned components."""

    def __init__(self, d_model=512, k_heads=4, v_heads=8, d=128, taps=4, rot=64):
        self.d_model, self.k_heads, self.v_heads, self.d, self.taps, self.rot = d_model, k_heads, v_heads, d, taps, rot
        self.keys, self.values = k_heads * d, v_heads * d
        self.conv = 2 * self.keys + self.values             # q, k, v
        self.cols = self.conv + self.values + 2 * v_heads   # then z, a, b


def random_weights(s, generator=None, device="cuda"):
    """One block's weights: projections bf16 [out][in], the rest f32."""

    def randn(*shape):
        return torch.randn(*shape, generator=generator, device=device)

    return {
        "norm": 1 + 0.1 * randn(s.d_model),
        "w_in": (randn(s.cols, s.d_model) * s.d_model ** -0.5).to(torch.bfloat16),
        "conv_w": randn(s.conv, s.taps) * 0.4,
        "conv_b": randn(s.conv) * 0.1,
        "A_log": torch.log(1 + 15 * torch.rand(s.v_heads, generator=generator, device=device)),
        "dt_bias": randn(s.v_heads) - 4,
        "inv_freq": 10000.0 ** (-torch.arange(0, s.rot, 2, device=device, dtype=torch.float32) / s.rot),
        "out_norm": 1 + 0.1 * randn(s.d),
        "w_out": (randn(s.d_model, s.values) * s.values ** -0.5).to(torch.bfloat16),
    }


class States:
    """The blocks' persistent states and the sequences' next positions."""

    def __init__(self, s, n_layers, batch, device="cuda"):
        self.conv = torch.zeros(n_layers, batch, s.conv, s.taps, device=device)
        self.delta = torch.zeros(n_layers, batch, s.v_heads, s.d, s.d, device=device)
        self.position = torch.zeros(batch, 1, dtype=torch.int64, device=device)


def _heads(t, first, heads, d):
    """Columns [first, first + heads d) of [B, T, cols] as [B, T, heads, d]."""
    return t[..., first:first + heads * d].unflatten(-1, (heads, d))


def prefill(s, layers, hidden, states):
    """hidden [B, T, d_model] f32 through the blocks in place, from and to states."""
    B, T, _ = hidden.shape
    bf = dict(dtype=torch.bfloat16, device=hidden.device)
    rows = hidden.view(B * T, s.d_model)
    h, proj = torch.empty(B * T, s.d_model, **bf), torch.empty(B, T, s.cols, **bf)
    u = torch.empty(B, T, s.conv, **bf)
    y, out = torch.empty(B, T, s.v_heads, s.d, **bf), torch.empty(B, T, s.v_heads, s.d, **bf)
    positions = states.position + torch.arange(T, device=hidden.device)
    q, k = _heads(u, 0, s.k_heads, s.d), _heads(u, s.keys, s.k_heads, s.d)
    v, z = _heads(u, 2 * s.keys, s.v_heads, s.d), _heads(proj, s.conv, s.v_heads, s.d)
    a = proj[..., s.conv + s.values:s.conv + s.values + s.v_heads]
    b = proj[..., s.conv + s.values + s.v_heads:]
    for n, w in enumerate(layers):
        m.mamba_rmsnorm(h, rows, w["norm"], EPS)
        m.mamba_linear_bf16(proj.view(B * T, s.cols), h, w["w_in"])
        m.mamba_conv1d_silu_prefill(u, proj[..., :s.conv], w["conv_w"], w["conv_b"], states.conv[n], states.conv[n])
        m.mamba_qk_norm_rotary(q, k, q, k, None, None, w["inv_freq"], positions, eps=EPS, l2=True)
        m.mamba_gated_delta_prefill(y, q, k, v, a, b, w["A_log"], w["dt_bias"], states.delta[n], states.delta[n])
        m.mamba_head_norm_gated(out, y, z, w["out_norm"], eps=EPS)
        m.mamba_linear_bf16(rows, out.view(B * T, s.values), w["w_out"], rows)
    states.position += T


class Decode:
    """One token through the blocks, recorded once: write hidden, launch(), read hidden."""

    def __init__(self, s, layers, states):
        self.s, self.layers, self.states = s, layers, states
        B, dev = states.position.shape[0], states.position.device
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.hidden = torch.zeros(B, s.d_model, device=dev)
        self.h = torch.empty(B, s.d_model, **bf)
        self.qkv, self.u, self.rest = (torch.empty(B, n, **bf) for n in (s.conv, s.conv, s.cols - s.conv))
        self.y, self.out = (torch.empty(B, s.v_heads, s.d, **bf) for _ in range(2))
        kept = [t.clone() for t in (states.conv, states.delta, states.position)]
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            self._token()  # once outside the recording, so that everything is loaded
        torch.cuda.current_stream(dev).wait_stream(side)
        for t, was in zip((states.conv, states.delta, states.position), kept):
            t.copy_(was)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._token()

    def _token(self):
        s, st = self.s, self.states
        q, k = (_heads(self.u[:, None], i * s.keys, s.k_heads, s.d) for i in range(2))
        v = _heads(self.u, 2 * s.keys, s.v_heads, s.d)
        z = _heads(self.rest, 0, s.v_heads, s.d)[:, None]
        a, b = (self.rest[:, s.values + i * s.v_heads:s.values + (i + 1) * s.v_heads] for i in range(2))
        for n, w in enumerate(self.layers):
            m.mamba_rmsnorm(self.h, self.hidden, w["norm"], EPS)
            m.mamba_linear_bf16(self.qkv, self.h, w["w_in"][:s.conv])
            m.mamba_linear_bf16(self.rest, self.h, w["w_in"][s.conv:])
            m.mamba_conv1d_silu_step(self.u, self.qkv, st.conv, n, w["conv_w"], w["conv_b"])
            m.mamba_qk_norm_rotary(q, k, q, k, None, None, w["inv_freq"], st.position, eps=EPS, l2=True)
            m.mamba_gated_delta_step_batched(self.y, q[:, 0], k[:, 0], v, a, b, w["A_log"], w["dt_bias"], st.delta, n)
            m.mamba_head_norm_gated(self.out[:, None], self.y[:, None], z, w["out_norm"], eps=EPS)
            m.mamba_linear_bf16(self.hidden, self.out.view(-1, s.values), w["w_out"], self.hidden)
        st.position += 1

    def launch(self):
        self.graph.replay()


def main():
    s, n_layers, B, T = Sizes(), 4, 8, 1000
    layers = [random_weights(s) for _ in range(n_layers)]
    states = States(s, n_layers, B)
    hidden = torch.randn(B, T, s.d_model, device="cuda")
    warm = States(s, n_layers, B)
    prefill(s, layers, hidden.clone(), warm)

    def timed(f):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        start.record()
        f()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end)

    ms = timed(lambda: prefill(s, layers, hidden, states))
    print(f"prompt: {n_layers} blocks, {B} x {T} tokens: {ms:.3f} ms")
    decode = Decode(s, layers, states)
    decode.hidden.copy_(hidden[:, -1])
    steps = 100
    ms = timed(lambda: [decode.launch() for _ in range(steps)])
    print(f"decode: {n_layers} blocks, batch {B}: {1e3 * ms / steps:.1f} us a token")
    faults = m.mamba_device_faults()
    assert faults == 0 and torch.isfinite(decode.hidden).all(), (faults, decode.hidden)


if __name__ == "__main__":
    main()
