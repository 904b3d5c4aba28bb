"""The operators of a training step run together, as they are used: a layer norm, the cross entropy of the output
projection (or the selective log-probabilities with a policy loss), their gradients, and the AdamW step that writes the
16-bit weights which the next step reads.

Each stage is checked against float64 (or, for AdamW, numpy's float32 bit for bit) on what the stage before it
gave, with the tolerances of the stages' own tests, so no error has to be carried through the chain.
"""
import numpy as np
import pytest
import torch

import adamw_reference as ref
import rl_post_loss_amd as rl
import synthetic
from test_adamw import DEV, f32_bits, same
from test_layer_norm import backward_case, forward_case
from test_linear_cross_entropy import IGNORE, U, check, expected

pytestmark = pytest.mark.gpu
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8)


class Head:
    """A layer norm and an output projection, float32 parameters with their bf16 copies, and an AdamW plan of them."""

    def __init__(self, H, V, state_dtype, seed):
        g = torch.Generator().manual_seed(seed)
        init = [1.0 + 0.1 * torch.randn(H, generator=g), 0.1 * torch.randn(H, generator=g),
                torch.randn(V, H, generator=g) * 2 / H ** 0.5, 0.1 * torch.randn(V, generator=g)]
        self.params = [t.to(DEV) for t in init]
        self.copies = [t.bfloat16() for t in self.params]
        self.plan = rl.adamw_plan(self.params, state_dtype=state_dtype, weight_decay=[0.0, 0.0, 0.1, 0.0],
                                  copies=self.copies)

    def forward_backward(self, x, targets):
        nw, nb, w, b = self.copies
        y, mean, rstd = rl.layer_norm_fwd(x, nw, nb)
        loss, dy, dw, db = rl.linear_cross_entropy(y, w, b, targets, z_loss=1e-3)
        dx, dnw, dnb = rl.layer_norm_bwd(dy, x, nw, mean, rstd)
        return dict(y=y, mean=mean, rstd=rstd, loss=loss, dy=dy, dx=dx, grads=[dnw, dnb, dw, db])


def batch(n, H, V, seed):
    g = torch.Generator().manual_seed(seed)
    y = torch.randint(0, V, (n,), generator=g)
    y[torch.rand(n, generator=g) < 0.3] = IGNORE
    return (1.5 * torch.randn(n, H, generator=g) + 0.5).bfloat16().to(DEV), y.to(DEV)


@pytest.mark.parametrize("state", [torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("n,H,V", [(1, 64, 300), (300, 128, 1500), (700, 72, 515)])
def test_steps_of_a_supervised_head(n, H, V, state):
    head = Head(H, V, state, seed=n)
    host = [t.cpu() for t in head.params]
    eight = state != torch.float32
    zeros = lambda d, f: [np.zeros(f(t.numel()), d) for t in host]  # noqa: E731
    m, v = zeros(np.float32, int), zeros(np.float32, int)
    mq, rq = zeros(np.uint8, int), zeros(np.uint8, int)
    ms, rs = zeros(np.float32, lambda k: (k + 255) // 256), zeros(np.float32, lambda k: (k + 255) // 256)
    p = [t.numpy().reshape(-1).copy() for t in host]
    for t in (1, 2, 3):
        x, targets = batch(n, H, V, 100 * t + n)
        before = [c.cpu() for c in head.copies]
        out = head.forward_backward(x, targets)
        rl.adamw_step(head.plan, out["grads"], step=t, seed=17, **HYPER)
        torch.cuda.synchronize()
        nw, nb, w, b = before
        forward_case(x.cpu(), nw, nb, 1e-5, (out["y"], out["mean"], out["rstd"]))
        want = expected({"h": out["y"].cpu(), "w": w, "b": b, "y": targets.cpu()}, 1e-3)
        check("loss", out["loss"], want["loss"])
        for name, g in (("grad_hidden", out["dy"]), ("grad_weight", out["grads"][2]), ("grad_bias", out["grads"][3])):
            check(name, g, want[name], U["bf16"])
        backward_case({"x": x.cpu(), "w": nw, "dy": out["dy"].cpu()}, out["mean"], out["rstd"],
                      (out["dx"], out["grads"][0], out["grads"][1]))
        k = ref.coefficients(HYPER["lr"], HYPER["betas"], HYPER["eps"], t)
        for i, g in enumerate(out["grads"]):
            g = g.float().cpu().numpy().reshape(-1)
            if eight:
                r0 = ref.decode(rq[i], rs[i])
                p[i], mm, r, _ = ref.step(p[i], g, ref.decode(mq[i], ms[i]), r0 * r0, k, head.plan.weight_decay[i])
                words = ref.random_words(17, t, i, g.size)
                mq[i], ms[i] = ref.encode(mm, words & np.uint64(0xFFFF), False)
                rq[i], rs[i] = ref.encode(r, words >> np.uint64(16), True)
                same("exp_avg", head.plan.exp_avg[i].view(-1), mq[i])
            else:
                p[i], m[i], _, v[i] = ref.step(p[i], g, m[i], v[i], k, head.plan.weight_decay[i])
                same("exp_avg", head.plan.exp_avg[i].view(-1), f32_bits(m[i]))
            same(f"param {i}", head.params[i].view(-1), f32_bits(p[i]))
            same(f"copy {i}", head.copies[i].view(-1), torch.from_numpy(p[i]).bfloat16())


@pytest.mark.parametrize("state", [torch.float32, torch.float8_e4m3fn])
def test_a_captured_step_replayed(state):
    """The whole step in one graph, replayed with new inputs, steps and rates, equals eager steps bit for bit."""
    n, H, V = 260, 64, 700
    a, b = Head(H, V, state, 1), Head(H, V, state, 1)
    x, targets = (t.clone() for t in batch(n, H, V, 1))
    step, lr = torch.ones(1, dtype=torch.int64, device=DEV), torch.tensor([3e-3], device=DEV)

    def run(head, x, targets, step, lr):
        out = head.forward_backward(x, targets)
        rl.adamw_step(head.plan, out["grads"], step=step, lr=lr, betas=(0.9, 0.99), seed=3)
        return out["loss"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(a, x, targets, step, lr)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    run(b, x, targets, 1, float(lr))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = run(a, x, targets, step, lr)
    for t in range(2, 6):
        nx, ny = batch(n, H, V, t)
        x.copy_(nx)
        targets.copy_(ny)
        step.fill_(t)
        lr.fill_(1e-3 * t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = run(b, nx, ny, t, float(lr))
        torch.cuda.synchronize()
        assert torch.equal(loss, want)
        for p, q in zip(a.params + a.copies + a.plan.exp_avg + a.plan.exp_avg_sq,
                        b.params + b.copies + b.plan.exp_avg + b.plan.exp_avg_sq):
            same(f"step {t}", p, q)


def test_autograd_of_the_norm_and_the_loss():
    """Both operators' autograd forms in one graph leave the gradients that the direct calls give."""
    head = Head(64, 400, torch.float32, 5)
    x, targets = batch(200, 64, 400, 9)
    out = head.forward_backward(x, targets)
    leaves = [t.clone().requires_grad_() for t in (x, *head.copies)]
    y = rl.layer_norm_autograd(*leaves[:3])
    loss = rl.linear_cross_entropy_autograd(y, leaves[3], leaves[4], targets, z_loss=1e-3)
    loss.backward()
    assert torch.equal(loss.detach(), out["loss"])
    for t, g in zip(leaves, (out["dx"], *out["grads"])):
        assert torch.equal(t.grad, g)


def test_step_of_a_policy_head():
    """Selective log-probabilities, the GRPO loss on them, their backward pass and the update of the projection: the
    float32 gradients go to the step as they are."""
    bs, T, H, V = 4, 50, 64, 600
    x = synthetic.chain_inputs(bs, T, H, V, "bf16", 0)
    d = {k: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for k, t in x.items()}
    w32 = d["weight"].float()
    w = d["weight"].clone()
    plan = rl.adamw_plan([w32], copies=[w], weight_decay=0.01)
    logp, lse = rl.selective_logprob_fwd(d["hidden"], w, d["bias"], d["targets"])
    lp = logp.view(bs, T)
    mask = torch.ones(bs, T, dtype=torch.bool, device=DEV)
    adv = torch.linspace(-1, 1, bs, device=DEV)
    _, g = rl.grpo_loss(lp, lp - 0.01, None, adv, mask)
    _, dw, _ = rl.selective_logprob_bwd(d["hidden"], w, d["bias"], d["targets"], lse, g.reshape(-1))
    before, w16 = w32.cpu().numpy().reshape(-1), w.clone()
    rl.adamw_step(plan, [dw], step=1, **HYPER)
    k = ref.coefficients(HYPER["lr"], HYPER["betas"], HYPER["eps"], 1)
    zero = np.zeros_like(before)
    p, m, _, v = ref.step(before, dw.cpu().numpy().reshape(-1), zero, zero, k, 0.01)
    same("param", w32.view(-1), f32_bits(p))
    same("copy", w.view(-1), torch.from_numpy(p).bfloat16())
    again, _ = rl.selective_logprob_fwd(d["hidden"], w, d["bias"], d["targets"])
    assert torch.isfinite(again).all() and not torch.equal(w, w16)


def test_operators_on_a_side_stream():
    """Called on another stream than the tensors were made on, with the workspaces and plan of the default one alive."""
    head = Head(64, 500, torch.float32, 2)
    x, targets = batch(150, 64, 500, 3)
    want = head.forward_backward(x, targets)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = head.forward_backward(x, targets)
        rl.adamw_step(head.plan, got["grads"], step=1, **HYPER)
    torch.cuda.synchronize()
    for a, b in zip([got["loss"], got["dy"], got["dx"], *got["grads"]], [want["loss"], want["dy"], want["dx"], *want["grads"]]):
        assert torch.equal(a, b)
