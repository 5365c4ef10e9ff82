"""The gated-delta-rule layer's operators, as they are measured: cases, inputs, plain forms and exact values.

  prefill    the gated delta rule over T tokens, state in and out
  step       the batched T = 1 step on one layer's state slab
  qk_norm    per-head norms of queries and keys with the position rotation
  head_norm  the per-head RMSNorm of the output with its SiLU(z) gate
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64


def listed():
    return [
        # one user, one token: a layer of 24 heads of 64 x 64 (d_inner 1536); latency counts
        dict(name="step_one", op="step", B=1, Hk=24, Hv=24, dk=64, dv=64, dtype="bf16"),
        # batched decode of the same layer, 128 sequences
        dict(name="step_batch", op="step", B=128, Hk=24, Hv=24, dk=64, dv=64, dtype="bf16"),
        # a wide layer's batched decode, key heads shared by two value heads, f32 activations
        dict(name="step_wide", op="step", B=128, Hk=16, Hv=32, dk=128, dv=128, dtype="f32"),
        # a short ragged prompt batch: T inside a chunk's second half
        dict(name="prefill_short", op="prefill", B=3, T=101, Hk=4, Hv=12, dk=128, dv=128, dtype="bf16", state=False),
        # one prompt on a small layer (d_inner 1536)
        dict(name="prefill_2k", op="prefill", B=1, T=2048, Hk=12, Hv=12, dk=128, dv=128, dtype="bf16", state=False),
        # f32 activations, heads of 64, an odd length, continuing from a state
        dict(name="prefill_f32", op="prefill", B=2, T=1777, Hk=12, Hv=24, dk=64, dv=64, dtype="f32", state=True),
        # long context, few heads, continuing from a state (d_inner 2048)
        dict(name="prefill_long", op="prefill", B=1, T=16384, Hk=16, Hv=16, dk=128, dv=128, dtype="bf16", state=True),
        # a batch of prompts on a large layer (d_inner 5120)
        dict(name="prefill_large", op="prefill", B=8, T=4096, Hk=40, Hv=40, dk=128, dv=128, dtype="bf16", state=False),
        # the decode step's queries and keys: 128 sequences at far, different positions
        dict(name="qk_decode", op="qk_norm", B=128, T=1, Hq=16, Hk=16, d=128, rot=64, dtype="bf16", l2=True,
             interleaved=False, weight=False, far=True),
        # a prompt batch's queries and keys, weighted norms, the whole head turned
        dict(name="qk_prompt", op="qk_norm", B=8, T=4096, Hq=16, Hk=8, d=128, rot=128, dtype="bf16", l2=False,
             interleaved=True, weight=True, far=False),
        # the decode step's output norm
        dict(name="norm_decode", op="head_norm", B=128, T=1, H=24, d=64, dtype="bf16"),
        # a prompt batch's output norm
        dict(name="norm_prompt", op="head_norm", B=8, T=4096, H=40, d=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "prefill", "prefill", "qk_norm", "head_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (128, 64), (96, 128), (128, 256), (72, 40)])
    Hk = _log_int(rng, 1, 24)
    Hv = Hk * rng.choice([1, 1, 2, 3])
    if op == "step":
        B = _log_int(rng, 1, 160)
        while B * Hv * dk * dv > 128 * 32 * 128 * 128:
            B = max(1, B // 2)
        return dict(op=op, B=B, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype)
    if op == "prefill":
        T = _log_int(rng, 1, 12000)
        B = _log_int(rng, 1, 8)
        while B * T * Hv * dk * dv > 8 * 4096 * 40 * 128 * 128 // 4:
            B, T = (B // 2, T) if B > 1 else (1, T // 2)
        return dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype, state=rng.random() < 0.5)
    T = rng.choice([1, _log_int(rng, 1, 4096)])
    B = _log_int(rng, 1, 128 if T == 1 else 8)
    d = rng.choice([64, 128, 128, 96, 80, 256])
    while B * T * (Hk + Hv) * d > 8 * 4096 * 40 * 128:
        T = T // 2
    if op == "qk_norm":
        rot = rng.choice([0, 32, d, d // 2])
        return dict(op=op, B=B, T=T, Hq=Hv, Hk=Hk, d=d, rot=rot, dtype=dtype, l2=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, weight=rng.random() < 0.5, far=rng.random() < 0.5)
    return dict(op=op, B=B, T=T, H=Hv, d=d, dtype=dtype)


def _inputs(case, seed):
    """The seeded inputs, on the GPU where there is one: names -> tensors."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + 17)
    dt = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    op, B = case["op"], case["B"]
    if op in ("step", "prefill"):
        T = case.get("T", 1)
        Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        lead = (B,) if op == "step" else (B, T)
        # queries and keys as the norms leave them (unit length); keys of a head share a direction in part, as a
        # model's do; v after conv + SiLU
        k = randn(*lead, Hk, dk) + 0.5 * randn(Hk, dk)
        q = randn(*lead, Hk, dk) + 0.5 * randn(Hk, dk)
        k = (k / k.square().sum(-1, keepdim=True).sqrt()).to(dt)
        q = (q / q.square().sum(-1, keepdim=True).sqrt()).to(dt)
        v = torch.nn.functional.silu(randn(*lead, Hv, dv)).to(dt)
        a = (0.5 * randn(*lead, Hv)).to(dt)
        b = randn(*lead, Hv).to(dt)
        # A in [1, 16), softplus(dt_bias) log-uniform in [1e-3, 0.1]: the usual initialisation
        A_log = torch.log(1 + 15 * rand(Hv))
        s = torch.exp(math.log(1e-3) + rand(Hv) * (math.log(0.1) - math.log(1e-3)))
        dt_bias = s + torch.log(-torch.expm1(-s))
        x = dict(q=q, k=k, v=v, a=a, b=b, A_log=A_log, dt_bias=dt_bias)
        if op == "step":
            x["state"] = 0.1 * randn(2, B, Hv, dv, dk)  # two layers' slabs; the step is the second's
        elif case["state"]:
            x["state_in"] = 0.1 * randn(B, Hv, dv, dk)
        return x
    T, d = case["T"], case["d"]
    if op == "qk_norm":
        x = dict(q=randn(B, T, case["Hq"], d).to(dt), k=randn(B, T, case["Hk"], d).to(dt))
        if case["weight"]:
            x["q_weight"], x["k_weight"] = 1 + 0.1 * randn(d), 1 + 0.1 * randn(d)
        rot = case["rot"]
        if rot:
            x["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float32) / rot)
        start = torch.randint(0, 1000000 if case["far"] else 1, (B, 1), generator=g, device=dev)
        x["positions"] = start + torch.arange(T, device=dev)
        return x
    return dict(y=randn(B, T, case["H"], d).to(dt), z=randn(B, T, case["H"], d).to(dt),
                weight=1 + 0.1 * randn(d))


def prepare(case, seed):
    x = _inputs(case, seed)
    op = case["op"]
    out = {}
    if op in ("step", "prefill"):
        out["y"] = torch.empty_like(x["v"])
        if op == "prefill":
            out["state_out"] = torch.empty(case["B"], case["Hv"], case["dv"], case["dk"], device=x["v"].device)
    elif op == "qk_norm":
        out["q_out"], out["k_out"] = torch.empty_like(x["q"]), torch.empty_like(x["k"])
    else:
        out["out"] = torch.empty_like(x["y"])
    return dict(case=case, x=x, out=out)


# ------------------------------------------------------------------ plain forms

def _gates(x):
    """log(alpha) and beta, [..., Hv] in 32 bits."""
    v = x["a"].float() + x["dt_bias"]
    softplus = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    return -torch.exp(x["A_log"]) * softplus, torch.sigmoid(x["b"].float())


def _plain_step(case, x):
    rep = case["Hv"] // case["Hk"]
    q = x["q"].float().repeat_interleave(rep, 1)
    k = x["k"].float().repeat_interleave(rep, 1)
    log_alpha, beta = _gates(x)
    state = x["state"][1]
    state.mul_(torch.exp(log_alpha)[..., None, None])
    u = beta[..., None] * (x["v"].float() - (state @ k[..., None])[..., 0])
    state.add_(u[..., None] * k[..., None, :])
    y = (state @ q[..., None])[..., 0] * case["dk"] ** -0.5
    return y.to(x["v"].dtype), state


def _plain_prefill(case, x):
    """Chunks of 64 tokens: the products inside a chunk for all chunks at once, the state from chunk to chunk."""
    B, T, Hk, Hv, dk, dv = (case[n] for n in ("B", "T", "Hk", "Hv", "dk", "dv"))
    rep, C = Hv // Hk, min(_CHUNK, case["T"])
    n = (T + C - 1) // C
    dev = x["v"].device

    def chunks(t):  # [B, T, H, d] -> [n, B, H, C, d], padded with zeros
        t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, n * C - T))
        return t.view(B, n, C, t.shape[2], t.shape[3]).permute(1, 0, 3, 2, 4)

    q = chunks(x["q"].float().repeat_interleave(rep, 2))
    k = chunks(x["k"].float().repeat_interleave(rep, 2))
    v = chunks(x["v"].float())
    log_alpha, beta = _gates(x)
    beta = chunks(beta[..., None])
    G = chunks(log_alpha[..., None]).double().cumsum(3)  # long sums: 64 bits
    decay = torch.tril(torch.exp((G - G.transpose(-1, -2)).clamp(max=0)).float())
    eG = torch.exp(G).float()
    A = torch.tril(beta * (k @ k.transpose(-1, -2)) * decay, -1)
    inv = torch.eye(C, device=dev).expand_as(A).clone()  # (I + A)^-1 by forward substitution
    for i in range(1, C):
        inv[..., i, :i] = -(A[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    U = inv @ (beta * v)
    W = inv @ (beta * eG * k)
    P = (q @ k.transpose(-1, -2)) * decay
    to_end = torch.exp(G[..., -1:, :] - G).float()
    S = x["state_in"].clone() if "state_in" in x else torch.zeros(B, Hv, dv, dk, device=dev)
    y = torch.empty(n, B, Hv, C, dv, device=dev)
    for c in range(n):
        new = U[c] - W[c] @ S.transpose(-1, -2)
        y[c] = (eG[c] * q[c]) @ S.transpose(-1, -2) + P[c] @ new
        S = eG[c][..., -1:, :] * S + new.transpose(-1, -2) @ (to_end[c] * k[c])
    y = y.permute(1, 0, 3, 2, 4).reshape(B, n * C, Hv, dv)[:, :T] * dk ** -0.5
    return y.to(x["v"].dtype), S


def _plain_qk_norm(case, x):
    rot, d = case["rot"], case["d"]
    if rot:
        theta = x["positions"].double()[..., None] * x["inv_freq"].double()  # far positions: 64 bits
        cos, sin = torch.cos(theta).float()[:, :, None], torch.sin(theta).float()[:, :, None]

    def one(t, w):
        f = t.float()
        ss = f.square().sum(-1, keepdim=True)
        f = f * torch.rsqrt((ss if case["l2"] else ss / d) + 1e-6)
        if w is not None:
            f = f * w
        if rot:
            if case["interleaved"]:
                lo, hi = f[..., 0:rot:2], f[..., 1:rot:2]
                turned = torch.stack((lo * cos - hi * sin, hi * cos + lo * sin), -1).flatten(-2)
            else:
                lo, hi = f[..., :rot // 2], f[..., rot // 2:rot]
                turned = torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1)
            f = torch.cat((turned, f[..., rot:]), -1)
        return f.to(t.dtype)

    return one(x["q"], x.get("q_weight")), one(x["k"], x.get("k_weight"))


def _plain_head_norm(case, x):
    y, z = x["y"].float(), x["z"].float()
    f = y * torch.rsqrt(y.square().sum(-1, keepdim=True) / case["d"] + 1e-5) * x["weight"]
    return (f * z / (1 + torch.exp(-z))).to(x["y"].dtype)


def run(state):
    case, x, out = state["case"], state["x"], state["out"]
    op = case["op"]
    if not own:
        if op == "step":
            return _plain_step(case, x)
        if op == "prefill":
            return _plain_prefill(case, x)
        if op == "qk_norm":
            return _plain_qk_norm(case, x)
        return _plain_head_norm(case, x)
    import selective_state_space_conv1d_gb300 as m
    if op == "step":
        m.mamba_gated_delta_step_batched(out["y"], x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"],
                                         x["state"], 1)
        return out["y"], x["state"][1]
    if op == "prefill":
        m.mamba_gated_delta_prefill(out["y"], x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"],
                                    x.get("state_in"), out["state_out"])
        return out["y"], out["state_out"]
    if op == "qk_norm":
        m.mamba_qk_norm_rotary(out["q_out"], out["k_out"], x["q"], x["k"], x.get("q_weight"), x.get("k_weight"),
                               x.get("inv_freq"), x["positions"], l2=case["l2"], interleaved=case["interleaved"])
        return out["q_out"], out["k_out"]
    m.mamba_head_norm_gated(out["out"], x["y"], x["z"], x["weight"])
    return out["out"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op, B, T = case["op"], case["B"], case.get("T", 1)
    if op in ("step", "prefill"):
        Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        state = B * Hv * dv * dk * 4
        n_state = 2 if op == "step" or case["state"] else 1
        per_token = (2 * Hk * dk + 2 * Hv * dv + 2 * Hv) * es
        # per token and head: S k, the rank-1 update, S q, the decay
        return dict(bytes=B * T * per_token + n_state * state + 8 * Hv, flops=B * T * Hv * 7 * dk * dv)
    if op == "qk_norm":
        n = B * T * (case["Hq"] + case["Hk"]) * case["d"]
        small = 8 * B * T + 2 * case["rot"] + (8 * case["d"] if case["weight"] else 0)
        return dict(bytes=2 * n * es + small, flops=8 * n)
    n = B * T * case["H"] * case["d"]
    return dict(bytes=3 * n * es + 4 * case["d"], flops=10 * n)


# ------------------------------------------------------------------ exact values

def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token, the norms and turns as complex products."""
    x = {n: t.double() for n, t in _inputs(case, seed).items()}
    op = case["op"]
    if op in ("step", "prefill"):
        Hk, Hv, dk = case["Hk"], case["Hv"], case["dk"]
        head = torch.arange(Hv, device=x["v"].device) // (Hv // Hk)
        seq = {n: (x[n][:, None] if op == "step" else x[n]) for n in ("q", "k", "v", "a", "b")}
        alpha = torch.exp(-torch.exp(x["A_log"]) * torch.logaddexp(seq["a"] + x["dt_bias"],
                                                                   torch.zeros_like(seq["a"])))
        beta = 1 / (1 + torch.exp(-seq["b"]))
        S = (x["state"][1] if op == "step" else x["state_in"].clone() if "state_in" in x else
             torch.zeros(case["B"], Hv, case["dv"], dk, device=head.device, dtype=torch.float64))
        y = torch.empty_like(seq["v"])
        for t in range(seq["v"].shape[1]):
            q, k = seq["q"][:, t, head], seq["k"][:, t, head]
            S *= alpha[:, t, :, None, None]
            err = seq["v"][:, t] - torch.matmul(S, k.unsqueeze(-1)).squeeze(-1)
            S.addcmul_((beta[:, t, :, None] * err).unsqueeze(-1), k.unsqueeze(-2))
            y[:, t] = torch.matmul(S, q.unsqueeze(-1)).squeeze(-1)
        y /= math.sqrt(dk)
        return (y[:, 0] if op == "step" else y), S
    if op == "qk_norm":
        rot = case["rot"]
        got = []
        for t, w in ((x["q"], x.get("q_weight")), (x["k"], x.get("k_weight"))):
            f = t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) / (1 if case["l2"] else case["d"]) + 1e-6)
            f = f if w is None else f * w
            if rot:
                r = f[..., :rot]
                pairs = r.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else r.unflatten(-1, (2, rot // 2)).mT
                angle = (x["positions"][..., None] * x["inv_freq"])[:, :, None]
                c = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle),
                                                                                               angle))
                f = torch.cat(((c if case["interleaved"] else c.mT).flatten(-2), f[..., rot:]), -1)
            got.append(f)
        return tuple(got)
    y, z = x["y"], x["z"]
    return y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + 1e-5) * x["weight"] * z * torch.sigmoid(z)
