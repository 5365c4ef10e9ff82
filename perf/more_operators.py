"""A token's path around the blocks' mixers, as it is measured: cases, inputs, plain forms and exact values.

  linear    a projection with 4-bit weights and group scales
  norm      the update of the residual stream after a block (norm after it, gate, scale) with the next block's norm
  logprobs  log probabilities of given tokens, entropy and the likeliest alternatives
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's token: the output projection of a large block, the residual added
        dict(name="linear_one", op="linear", M=1, N=2560, K=5120, group=128, zeros=False, scales="bf16", out="f32",
             residual=True),
        # four users' tokens to a vocabulary of 50000: the head
        dict(name="linear_head", op="linear", M=4, N=50000, K=2560, group=128, zeros=False, scales="bf16", out="f32",
             residual=False),
        # a ragged projection, 23 tokens in flight, fine groups with zero points
        dict(name="linear_ragged", op="linear", M=23, N=1003, K=1000, group=32, zeros=True, scales="f32", out="bf16",
             residual=False),
        # batched decode: the input projection of a large block, 128 sequences
        dict(name="linear_batch", op="linear", M=128, N=10240, K=2560, group=64, zeros=True, scales="bf16",
             out="bf16", residual=False),
        # a batch of prompts through the same projection
        dict(name="linear_prompt", op="linear", M=8192, N=10240, K=2560, group=128, zeros=False, scales="bf16",
             out="bf16", residual=False),
        # one user's token between two blocks, norms before and after, a scale per channel
        dict(name="norm_one", op="norm", B=1, T=1, D=2560, y="bf16", out="bf16", post=True, gate="channel",
             gate_dtype="f32"),
        # batched decode of a small model, the residual scale alone
        dict(name="norm_decode", op="norm", B=128, T=1, D=768, y="bf16", out="bf16", post=False, gate="none",
             gate_dtype="f32"),
        # a batch of prompts, norms before and after, the gate of each sequence
        dict(name="norm_prompt", op="norm", B=8, T=4096, D=2560, y="bf16", out="bf16", post=True, gate="sequence",
             gate_dtype="bf16"),
        # one user's token: its probability and five alternatives
        dict(name="logprobs_one", op="logprobs", M=1, V=50000, dtype="f32", top=5, masked=0.0),
        # a constrained answer: most of an odd vocabulary masked out
        dict(name="logprobs_masked", op="logprobs", M=33, V=32003, dtype="f32", top=8, masked=0.9),
        # batched decode, a large vocabulary, twenty alternatives
        dict(name="logprobs_decode", op="logprobs", M=128, V=128000, dtype="bf16", top=20, masked=0.0),
        # scoring a batch of prompts: the given tokens and the entropy
        dict(name="logprobs_score", op="logprobs", M=8192, V=50000, dtype="bf16", top=0, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "logprobs"])
    if op == "linear":
        M = rng.choice([_log_int(rng, 1, 16), _log_int(rng, 1, 256), _log_int(rng, 1, 8192)])
        N, K = _log_int(rng, 256, 50000), _log_int(rng, 48, 6000)
        if rng.random() < 0.7:
            N, K = max(16, N // 16 * 16), max(64, K // 32 * 32)
        while M * N * K > 8192 * 10240 * 2560 or N * K > 50000 * 2560:
            M, N = max(1, M // 2), N // 2
        return dict(op=op, M=M, N=N, K=K, group=rng.choice([32, 64, 128, 128]), zeros=rng.random() < 0.5,
                    scales=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    residual=rng.random() < 0.3)
    if op == "norm":
        T = rng.choice([1, _log_int(rng, 1, 4096)])
        B, D = _log_int(rng, 1, 128 if T == 1 else 8), _log_int(rng, 96, 9000)
        if rng.random() < 0.7:
            D = D // 16 * 16
        while B * T * D > 8 * 4096 * 2560:
            T = T // 2
        return dict(op=op, B=B, T=T, D=D, y=rng.choice(["bf16", "bf16", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f32"]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "sequence", "token"]),
                    gate_dtype=rng.choice(["bf16", "f32"]))
    M, V = _log_int(rng, 1, 8192), _log_int(rng, 100, 260000)
    dtype = rng.choice(["bf16", "f32"])
    while M * V * (2 if dtype == "bf16" else 4) > 8192 * 50000 * 2:
        M = M // 2
    top = rng.choice([0, 1, rng.randint(1, 32)])
    if M > 1024:
        top = 0
    return dict(op=op, M=M, V=V, dtype=dtype, top=top, masked=rng.choice([0.0, 0.0, 0.5, 0.95]))


def _quantize(w, group, zeros, scale_dtype):
    """Weights [N, K] to 4 bits: values 0..15 [N, K], scales and zero points [N, groups] (None: 8)."""
    N, K = w.shape
    G = (K + group - 1) // group
    p = torch.nn.functional.pad(w, (0, G * group - K)).view(N, G, group)
    if zeros:
        lo, hi = p.amin(-1).clamp(max=0), p.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).clamp(min=1e-8).to(scale_dtype)
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s = (p.abs().amax(-1) / 7).clamp(min=1e-8).to(scale_dtype)
        z = torch.full_like(s, 8, dtype=torch.float32)
    q = (torch.round(p / s.float()[..., None]) + z[..., None]).clamp(0, 15)
    return q.view(N, G * group)[:, :K].to(torch.uint8), s, z.to(torch.uint8) if zeros else None


def _inputs(case, seed):
    """The seeded inputs, on the GPU where there is one: names -> tensors."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + 29)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        q, s, z = _quantize(randn(N, K) * K ** -0.5, case["group"], case["zeros"], _DT[case["scales"]])
        rows = torch.nn.functional.pad(q, (0, (K + 31) // 32 * 32 - K))
        # activations in rows of whole 16 bytes, as a program keeps them for tensor copies
        a = randn(M, (K + 7) // 8 * 8).to(torch.bfloat16)[:, :K]
        x = dict(a=a, q=rows[:, 0::2] | (rows[:, 1::2] << 4), scales=s)
        if z is not None:
            x["zeros"] = z
        if case["residual"]:
            x["residual"] = randn(M, N)
        return x
    if op == "norm":
        B, T, D = case["B"], case["T"], case["D"]
        # a residual stream that has grown over some blocks, a block's output of another size
        x = dict(x=3 * randn(B, T, D), y=(0.7 * randn(B, T, D)).to(_DT[case["y"]]), pre=1 + 0.1 * randn(D))
        if case["post"]:
            x["post"] = 1 + 0.1 * randn(D)
        shape = dict(none=None, channel=(D,), sequence=(B, D), token=(B, T, D))[case["gate"]]
        if shape:
            x["gate"] = (0.5 + 0.3 * randn(*shape)).to(_DT[case["gate_dtype"]])
        return x
    M, V = case["M"], case["V"]
    # a model's logits: a bulk, and for every row a few tokens that stand out
    logits = 2 * randn(M, V)
    likely = torch.randint(0, V, (M, 16), generator=g, device=dev)
    logits.scatter_add_(1, likely, 8 * rand(M, 16))
    if case["masked"]:
        mask = rand(M, V) < case["masked"]
        logits.masked_fill_(mask.scatter_(1, likely, False), float("-inf"))
    tokens = likely[torch.arange(M, device=dev), torch.randint(0, 16, (M,), generator=g, device=dev)]
    return dict(logits=logits.to(_DT[case["dtype"]]), tokens=tokens)


_SCALE = 0.75  # of a block's update: the residual scale


def prepare(case, seed):
    x = _inputs(case, seed)
    dev = next(iter(x.values())).device
    out = {}
    if case["op"] == "linear":
        out["c"] = torch.empty(case["M"], case["N"], device=dev, dtype=_DT[case["out"]])
    elif case["op"] == "norm":
        out["x"] = torch.empty_like(x["x"])
        out["out"] = torch.empty_like(x["x"], dtype=_DT[case["out"]])
    else:
        M, top = case["M"], case["top"]
        out["logprob"], out["entropy"] = torch.empty(M, device=dev), torch.empty(M, device=dev)
        if top:
            top = min(top, case["V"])
            out["top_logprob"] = torch.empty(M, top, device=dev)
            out["top_id"] = torch.empty(M, top, device=dev, dtype=torch.int64)
    return dict(case=case, x=x, out=out)


# ------------------------------------------------------------------ plain forms

def _plain_linear(case, x):
    K, group = case["K"], case["group"]
    q = torch.stack((x["q"] & 15, x["q"] >> 4), -1).flatten(1)[:, :K].float()
    q = q - (x["zeros"].float().repeat_interleave(group, 1)[:, :K] if "zeros" in x else 8.0)
    c = x["a"].float() @ (q * x["scales"].float().repeat_interleave(group, 1)[:, :K]).T
    if "residual" in x:
        c = c + x["residual"]
    return c.to(_DT[case["out"]])


def _plain_norm(case, x):
    n = x["y"].float()
    if "post" in x:
        n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + 1e-5) * x["post"]
    if "gate" in x:
        gate = x["gate"].float()
        n = n * (gate[:, None] if case["gate"] == "sequence" else gate)
    s = x["x"] + _SCALE * n
    h = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-5) * x["pre"]
    return s, h.to(_DT[case["out"]])


def _plain_logprobs(case, x):
    f = x["logits"].float()
    d = f - f.amax(-1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(-1)
    log_total = torch.log(total)
    logprob = d.gather(1, x["tokens"][:, None])[:, 0] - log_total
    entropy = log_total - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(-1) / total
    if not case["top"]:
        return logprob, entropy
    value, index = torch.sort(f, dim=-1, descending=True, stable=True)
    top = min(case["top"], case["V"])
    return logprob, entropy, value[:, :top] - f.amax(-1, keepdim=True) - log_total[:, None], index[:, :top].contiguous()


def run(state):
    case, x, out = state["case"], state["x"], state["out"]
    op = case["op"]
    if not own:
        return dict(linear=_plain_linear, norm=_plain_norm, logprobs=_plain_logprobs)[op](case, x)
    import selective_state_space_conv1d_gb300 as m
    if op == "linear":
        m.mamba_linear_w4(out["c"], x["a"], x["q"], x["scales"], x.get("zeros"), x.get("residual"),
                          group=case["group"])
        return out["c"]
    if op == "norm":
        m.mamba_block_norm(out["x"], out["out"], x["x"], x["y"], x["pre"], x.get("post"), x.get("gate"), scale=_SCALE)
        return out["x"], out["out"]
    m.mamba_token_logprobs(out["logprob"], out["entropy"], out.get("top_logprob"), out.get("top_id"), x["logits"],
                           x["tokens"])
    return tuple(out.values())


def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        groups = (K + case["group"] - 1) // case["group"]
        weights = N * ((K + 1) // 2) + N * groups * (size[case["scales"]] + (1 if case["zeros"] else 0))
        rows = 2 * M * K + M * N * (size[case["out"]] + (4 if case["residual"] else 0))
        return dict(bytes=weights + rows, flops=2 * M * N * K)
    if op == "norm":
        B, T, D = case["B"], case["T"], case["D"]
        gate = dict(none=0, channel=D, sequence=B * D, token=B * T * D)[case["gate"]] * size[case["gate_dtype"]]
        n = B * T * D
        return dict(bytes=n * (8 + size[case["y"]] + size[case["out"]]) + gate + 4 * D * (1 + case["post"]),
                    flops=n * (6 + 4 * case["post"]))
    M, V, top = case["M"], case["V"], case["top"]
    return dict(bytes=M * V * size[case["dtype"]] + M * (16 + 12 * top), flops=5 * M * V)


# ------------------------------------------------------------------ exact values

def exact(case, seed):
    """The definitions in 64 bits: sums per group, norms by lengths, probabilities by logsumexp and ranks by counting."""
    x = _inputs(case, seed)
    op = case["op"]
    if op == "linear":
        M, N, K, group = (case[n] for n in ("M", "N", "K", "group"))
        c = x["residual"].double() if "residual" in x else torch.zeros(M, N, dtype=torch.float64, device=x["a"].device)
        for g in range(x["scales"].shape[1]):
            lo, hi = g * group, min(K, (g + 1) * group)
            k = torch.arange(lo, hi, device=c.device)
            q = (x["q"][:, k // 2].int() >> (4 * (k % 2)).int()) % 16
            w = q.double() - (x["zeros"][:, g:g + 1].double() if "zeros" in x else 8)
            c += torch.einsum("mk,nk->mn", x["a"][:, lo:hi].double(), w) * x["scales"][:, g].double()
        return c
    x = {n: t.double() if t.is_floating_point() else t for n, t in x.items()}
    if op == "norm":
        D = case["D"]

        def unit(t):
            return t / torch.sqrt(torch.linalg.vector_norm(t, dim=-1, keepdim=True) ** 2 / D + 1e-5)

        update = unit(x["y"]) * x["post"] if "post" in x else x["y"]
        if "gate" in x:
            shape = dict(channel=(1, 1, D), sequence=(case["B"], 1, D), token=update.shape)[case["gate"]]
            update = update * x["gate"].reshape(shape)
        s = torch.add(x["x"], update, alpha=_SCALE)
        return s, unit(s) * x["pre"]
    logprob, entropy, tops, ids = [], [], [], []
    top = min(case["top"], case["V"])
    step = max(1, (1 << 26) // case["V"])
    for lo in range(0, case["M"], step):
        rows = x["logits"][lo:lo + step]
        lp = rows - torch.logsumexp(rows, -1, keepdim=True)
        logprob.append(lp.gather(1, x["tokens"][lo:lo + step, None])[:, 0])
        entropy.append(-torch.special.xlogy(lp.exp(), lp.exp()).sum(-1))
        free = torch.ones_like(rows, dtype=torch.bool)
        for _ in range(top):
            best = rows.masked_fill(~free, -math.inf).amax(-1, keepdim=True)
            first = (rows == best) & free
            index = (first.int().cumsum(-1) == 0).sum(-1, keepdim=True)  # how many stand before the first
            tops.append(lp.gather(1, index))
            ids.append(index)
            free.scatter_(1, index, False)
    logprob, entropy = torch.cat(logprob), torch.cat(entropy)
    if not top:
        return logprob, entropy
    n = len(tops) // top
    rows = lambda parts: torch.cat([torch.cat(parts[i * top:(i + 1) * top], 1) for i in range(n)])  # noqa: E731
    return logprob, entropy, rows(tops), rows(ids)
