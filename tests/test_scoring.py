"""The scoring operators and those around the gradients run together, as they are used.

A scoring pass: a residual stream and a block's output to an 8-bit norm, an 8-bit projection, and the log-probs, entropies and
alternatives of its logits.  A policy step: the norm, the logits, their log-probs with an entropy bonus under a policy
loss, the gradients back to the stream and the projection, and an AdamW step with the clipping factor.  Each stage is
checked against float64 on what the stage before it gave, with the tolerances of the stages' own tests.
"""
import pytest
import torch

import rl_post_loss_amd as rl
import test_fp8_linear as fp8
import test_grad_norm as norms
import test_rms_norm as rms
import test_token_logprobs as token

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Head:
    """A final norm's weight and an output projection in 8 bits."""

    def __init__(self, H, V, seed):
        g = torch.Generator().manual_seed(seed)
        self.norm = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().to(DEV)
        self.weight = (torch.randn(V, H, generator=g) * 3 / H ** 0.5).bfloat16().to(DEV)
        self.q, self.scale = rl.fp8_quantize(self.weight, block_rows=128)

    def score(self, x, residual, targets, mask, top_k):
        q, scale, rstd, stream = rl.rms_norm_fp8(x, self.norm, residual)
        logits = rl.fp8_linear(q, scale, self.q, self.scale)
        return dict(q=q, scale=scale, rstd=rstd, stream=stream, logits=logits,
                    out=rl.token_logprobs_fwd(logits, targets, mask, temperature=0.9, top_k=top_k))


def batch(shape, H, V, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, H, generator=g).bfloat16().to(DEV), 2 * torch.randn(*shape, H, generator=g).bfloat16().to(DEV),
            torch.randint(0, V, shape, generator=g).to(DEV), (torch.rand(*shape, generator=g) < 0.7).to(DEV))


@pytest.mark.parametrize("shape,H,V,top_k", [((1,), 256, 1000, 20), ((3, 40), 384, 2051, 5), ((2, 300), 144, 515, 1),
                                             ((700,), 1024, 5003, 0)])
def test_a_scoring_pass(shape, H, V, top_k):
    head = Head(H, V, seed=V)
    x, r, y, mask = batch(shape, H, V, 3)
    s = head.score(x, r, y, mask, top_k)
    rms.forward_case(x.cpu(), head.norm.cpu(), r.cpu(), 1e-6, s["rstd"], s["stream"], q=s["q"].cpu(), scale=s["scale"])
    w, ws = fp8.quantised(head.weight.cpu(), 128)
    assert torch.equal(head.scale.cpu(), ws) and torch.equal(head.q.cpu().view(torch.uint8), w.view(torch.uint8))
    n = x.numel() // H
    fp8.product_case(s["q"].cpu().view(n, H), s["scale"].cpu().view(n, -1), w, ws, None, s["logits"].view(n, V))
    flat = [None if t is None else t.reshape(n, *t.shape[len(shape):]) for t in s["out"]]
    token.forward_case(s["logits"].cpu().view(n, V), y.cpu().view(n), 0.9, flat, top_k, mask.cpu().view(n))


def test_a_captured_scoring_pass():
    head = Head(512, 3001, seed=1)
    x, r, y, mask = batch((33,), 512, 3001, 5)
    head.score(x, r, y, mask, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = head.score(x, r, y, mask, 8)
    for i in range(3):
        for t, new in zip((x, r, y, mask), batch((33,), 512, 3001, 10 + i)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        ref = head.score(x, r, y, mask, 8)
        assert torch.equal(s["logits"], ref["logits"]) and all(torch.equal(a, b) for a, b in zip(s["out"], ref["out"]))


def test_two_scoring_passes_at_once():
    """Each on a stream of its own, with workspaces of their own: the bits of one after the other."""
    passes = []
    for rows, H, V, top_k in ((700, 1024, 20011, 5), (33, 2048, 70001, 64)):
        head, inputs = Head(H, V, seed=V), batch((rows,), H, V, 7)
        passes.append((head, inputs, top_k, head.score(*inputs, top_k), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for head, inputs, top_k, _, stream in passes:
            with torch.cuda.stream(stream):
                got.append([head.score(*inputs, top_k) for _ in range(2)])
        torch.cuda.synchronize()
        for results, (_, _, _, ref, _) in zip(got, passes):
            for s in results:
                assert torch.equal(s["logits"], ref["logits"]) and torch.equal(s["q"].view(torch.uint8), ref["q"].view(torch.uint8))
                assert all(torch.equal(a, b) for a, b in zip(s["out"], ref["out"]))


@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
def test_a_policy_step_with_an_entropy_bonus(max_norm):
    """Gradients of every stage through the autograd forms, clipped by the factor that the optimizer takes."""
    B, T, H, V = 4, 24, 128, 515
    g = torch.Generator().manual_seed(0)
    x, r, y, mask = batch((B, T), H, V, 7)
    params = [(1 + 0.1 * torch.randn(H, generator=g)).to(DEV), (torch.randn(V, H, generator=g) * 3 / H ** 0.5).to(DEV)]
    copies = [p.bfloat16() for p in params]
    plan = rl.adamw_plan(params, copies=copies)
    old = [t.clone() for t in params]
    adv = torch.randn(B, generator=g).to(DEV)
    w, proj = (c.clone().requires_grad_() for c in copies)
    r.requires_grad_()
    h, stream = rl.rms_norm_autograd(x, w, r)
    logits = h[:, :-1] @ proj.t()
    logits.retain_grad()
    t, m = y[:, 1:].contiguous(), mask[:, 1:].contiguous()
    logp, entropy = rl.token_logprobs_autograd(logits, t, m)
    before = rl.token_logprobs_fwd(logits.detach(), t, m)[0]
    loss = rl.bnpo_loss_autograd(logp, before, None, adv, m) - 0.01 * (entropy * m).sum() / m.sum()
    loss.backward()
    # the policy loss at equal log-probs has the gradient -A / N; the bonus -0.01 / N
    N = int(m.sum())
    out = rl.token_logprobs_fwd(logits.detach(), t, m)
    flat = logits.detach().cpu().view(-1, V)
    on = m.cpu().view(-1)
    gl = (-adv[:, None].expand(B, T - 1) / N).cpu().reshape(-1)
    gh = torch.full_like(gl, -0.01 / N)
    token.backward_case(flat[on], t.cpu().view(-1)[on], 1.0, out[1].cpu().view(-1)[on], out[2].cpu().view(-1)[on], gl[on], gh[on],
                        logits.grad.view(-1, V)[on.to(DEV)])
    assert (logits.grad.view(-1, V)[~on.to(DEV)] == 0).all() and stream.shape == r.shape
    grads = [w.grad, proj.grad]
    norm, scale = rl.grad_norm(grads, max_norm=max_norm)
    want = norms.norm_of(grads)
    norms.near(norm, want, 1.01)
    norms.near(scale, min(1.0, max_norm / (want + 1e-6)), 4)
    rl.adamw_step(plan, grads, step=1, lr=1e-2, grad_scale=scale)
    for p, q, c in zip(old, params, copies):
        assert not torch.equal(p, q) and torch.equal(c, q.bfloat16())
    assert r.grad is not None and r.grad.isfinite().all()
