"""A token's path from the blocks to its log probability, stage by stage: each call's output
against 64 bits on what the call was given, so that every stage has the bound of its own
test (test_layer_w4 runs the path as one, where roundings of one stage spread in the next).
"""
import pytest
import torch

import selective_state_space_conv1d_gb300 as m
import test_block_norm as norm
import test_linear_w4 as linear
import test_token_logprobs as logprobs
from test_layer_w4 import block_by_calls, block_weights


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (1, 33), (2, 90)])
@pytest.mark.parametrize("captured", [False, True])
def test_every_stage_of_the_path(cuda_lib, B, T, captured):
    dm, V, M = 64, 501, B * T
    g = torch.Generator().manual_seed(5)
    blocks = [block_weights(20 + i, device="cuda")[0] for i in range(2)]
    head = m.quantize_w4(torch.randn(V, dm, generator=g).cuda() * 0.3, 64, zeros=True)
    branch = m.quantize_w4(torch.randn(dm, dm, generator=g).cuda() * dm ** -0.5, 32)
    post, pre = ((1 + 0.1 * torch.randn(dm, generator=g)).cuda() for _ in range(2))
    gate = torch.rand(B, dm, generator=g).cuda()
    x0 = torch.randn(B, T, dm, generator=g).cuda()
    tokens = torch.randint(0, V, (M,), generator=g).cuda()
    hidden, summed = x0.clone(), torch.empty_like(x0)
    n, y, out = (torch.empty(B, T, dm, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    logits, lp, h = (torch.empty(*s, device="cuda") for s in ((M, V), (M,), (M,)))
    tl, ti = torch.empty(M, 4, device="cuda"), torch.empty(M, 4, device="cuda", dtype=torch.int64)

    def call():
        for w in blocks:
            m.mamba_layer_prefill(hidden, w)
        m.mamba_rmsnorm(n.view(M, dm), hidden.view(M, dm), pre)
        m.mamba_linear_w4(y.view(M, dm), n.view(M, dm), *branch[:3], group=branch.group)
        m.mamba_block_norm(summed, out, hidden, y, pre, post, gate, scale=0.5)
        m.mamba_linear_w4(logits, out.view(M, dm), *head[:3], group=head.group)
        m.mamba_token_logprobs(lp, h, tl, ti, logits, tokens)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        hidden.copy_(x0)
        graph.replay()
    else:
        call()
    torch.cuda.synchronize()

    want = x0.clone()
    for w in blocks:
        zero = lambda c: torch.zeros(B, 128, c, device="cuda")  # noqa: E731
        block_by_calls(want, w, zero(4), zero(16))
    assert torch.equal(hidden, want)
    # the norm of the stream: block_norm's bound with nothing added
    norm.check(n, norm.reference(hidden, torch.zeros_like(hidden), pre, None, None, 1.0)[1])
    cpu = lambda w: [None if t is None else t.cpu() for t in w[:3]]  # noqa: E731
    linear.check(y.view(M, dm), *linear.reference(n.view(M, dm), *cpu(branch), branch.group), dm)
    for got, ref in zip((summed, out), norm.reference(hidden, y, pre, post, gate[:, None], 0.5)):
        norm.check(got, ref)
    linear.check(logits, *linear.reference(out.view(M, dm), *cpu(head), head.group), dm)
    ref, ref_h, log_s1 = logprobs.reference(logits)
    rel, U = (V / 256 + 110) * logprobs.U, logprobs.U
    at = ref.gather(1, tokens.cpu()[:, None])[:, 0]
    logprobs.close(lp, at, rel + 4 * U * (log_s1 + at.abs()), "logprob")
    logprobs.close(h, ref_h, rel + 4 * U * log_s1 + 4 * rel * (ref_h - log_s1).abs(), "entropy")
    order = torch.sort(logits.cpu(), dim=-1, descending=True, stable=True).indices[:, :4]
    best = ref.gather(1, order)
    logprobs.close(tl, best, rel + 4 * U * (log_s1[:, None] + best.abs()), "top")
    assert torch.equal(ti.cpu(), order)
    assert m.mamba_device_faults() == 0
