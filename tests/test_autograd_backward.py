"""What the autograd forms do in a backward pass besides the gradients: on the CPU, with the operators' bodies replaced
by their formulas in torch (the ops, their fakes and their autograd formulas are the package's own)."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import rl_post_loss_amd as rl
import rl_post_loss_amd.autograd as ag


def ce_formula(hidden, weight, bias, targets, *, ignore_index=-100, z_loss=0.0, reduction="mean", need_hidden=True,
               need_weight=True, need_bias=True, weight_grad_dtype=None, hidden_grad_dtype=None, **_):
    h, w, keep = hidden.double(), weight.double(), targets != ignore_index
    z = h @ w.t() if bias is None else h @ w.t() + bias.double()
    scale = keep.double() / (keep.sum().clamp(min=1) if reduction == "mean" else 1)
    at = torch.where(keep, targets, 0)[:, None]
    lse = torch.logsumexp(z, 1)
    loss = (scale * (lse - z.gather(1, at)[:, 0] + z_loss * lse ** 2)).sum()
    dz = (1 + 2 * z_loss * lse)[:, None] * torch.exp(z - lse[:, None])
    dz = scale[:, None] * dz.scatter_add(1, at, -torch.ones_like(scale)[:, None])
    wdt = weight_grad_dtype or hidden.dtype
    return (loss.float(), (dz @ w).to(hidden_grad_dtype or hidden.dtype) if need_hidden else None,
            (dz.t() @ h).to(wdt) if need_weight else None, dz.sum(0).to(wdt) if need_bias and bias is not None else None)


def norm_formula(x, weight=None, bias=None, *, eps=1e-5):
    mean = x.float().mean(-1)
    rstd = (x.float().var(-1, unbiased=False) + eps).rsqrt()
    y = (x.float() - mean[..., None]) * rstd[..., None]
    y = y if weight is None else y * weight.float()
    return (y if bias is None else y + bias.float()).to(x.dtype), mean, rstd


def norm_backward_formula(grad_y, x, weight, mean, rstd, *, need_x=True, need_weight=True, need_bias=True, **_):
    h = (x.float() - mean[..., None]) * rstd[..., None]
    g = grad_y.float() if weight is None else grad_y.float() * weight.float()
    dx = rstd[..., None] * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    rows = tuple(range(x.dim() - 1))
    wdt = x.dtype if weight is None else weight.dtype
    return (dx.to(x.dtype) if need_x else None,
            (grad_y.float() * h).sum(rows).to(wdt) if need_weight and weight is not None else None,
            grad_y.float().sum(rows).to(wdt) if need_bias else None)


def policy_formula(op, fused, lp, *rest):
    return (lp.detach().float() ** 2).sum(), 2 * lp.detach()


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(ag, "linear_cross_entropy", ce_formula)
    monkeypatch.setattr(ag, "linear_cross_entropy_fwd", lambda *a, **k: ce_formula(*a, **k)[0])
    monkeypatch.setattr(ag, "layer_norm_fwd", norm_formula)
    monkeypatch.setattr(ag, "layer_norm_bwd", norm_backward_formula)
    monkeypatch.setattr(ag, "_policy", policy_formula)


class Made(TorchDispatchMode):
    """Sizes of the tensors filled with zeros while the mode is on."""

    def __init__(self):
        super().__init__()
        self.zeros = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "zero" in func._schema.name:
            self.zeros.append(out.numel())
        return out


def case(n=6, H=8, V=40, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    return r(n, H), r(V, H), r(V), torch.randint(0, V, (n,), generator=g)


def test_no_tensor_of_zeros_stands_for_an_unused_gradient(on_cpu):
    """The ops return the gradients beside the loss; their own gradients, which nobody asks for, are not made up."""
    h, w, b, y = case()
    h, w, b = (t.requires_grad_() for t in (h, w, b))
    loss = rl.linear_cross_entropy_autograd(h, w, b, y)
    with Made() as made:
        loss.backward()
    assert not made.zeros
    assert h.grad is not None and w.grad is not None and b.grad is not None
    x = torch.randn(5, 7, requires_grad=True)
    out = rl.layer_norm_autograd(x)
    with Made() as made:
        out.backward(torch.ones(5, 7))
    assert not made.zeros
    lp = torch.randn(3, 4, requires_grad=True)
    loss = rl.bnpo_loss_autograd(lp, lp.detach(), None, torch.ones(3), torch.ones(3, 4, dtype=torch.bool))
    with Made() as made:
        loss.backward()
    assert not made.zeros and torch.equal(lp.grad, 2 * lp.detach())


@pytest.mark.gpu
def test_memory_of_the_backward_pass():
    """Beside what the forward pass left, a backward pass takes the gradients it returns: less than half a projection
    more than the one gradient wanted."""
    n, H, V = 64, 512, 32768
    r = lambda *s: torch.randn(*s, device="cuda:0").bfloat16()  # noqa: E731
    h, w, y = r(n, H), r(V, H).requires_grad_(), torch.randint(0, V, (n,), device="cuda:0")
    loss = rl.linear_cross_entropy_autograd(h, w, None, y)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    loss.backward()
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < 3 * V * H
    assert torch.equal(w.grad, rl.linear_cross_entropy(h, w, None, y)[2])


def test_second_derivatives_are_refused(on_cpu):
    """The gradients are values, not functions of the inputs: asking for their own gradient raises."""
    h, w, b, y = case()
    h, w, b = (t.requires_grad_() for t in (h, w, b))
    for wanted in (h, w, b):
        (d,) = torch.autograd.grad(rl.linear_cross_entropy_autograd(h, w, b, y), wanted, create_graph=True)
        with pytest.raises(RuntimeError, match="linear_cross_entropy_autograd.*first derivatives"):
            d.float().square().sum().backward()
    lp = torch.randn(3, 4, requires_grad=True)
    for op in ("bnpo", "grpo"):
        loss = getattr(rl, f"{op}_loss_autograd")(lp, lp.detach(), None, torch.ones(3), torch.ones(3, 4, dtype=torch.bool))
        (d,) = torch.autograd.grad(loss, lp, create_graph=True)
        with pytest.raises(RuntimeError, match=f"{op}_loss_autograd.*first derivatives"):
            torch.autograd.grad(d.sum(), lp)
    x = torch.randn(5, 7, requires_grad=True)
    (d,) = torch.autograd.grad(rl.layer_norm_autograd(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        d.square().sum().backward()
    with pytest.raises(RuntimeError, match="layer_norm_autograd"):
        torch.ops.rlpl.layer_norm(x, None, None, 1e-5)[1].sum().backward()    # the statistics


def test_a_gradient_with_respect_to_the_factor_of_the_loss(on_cpu):
    """d (s * loss) / d hidden is linear in s, and its gradient in s is the loss's own."""
    h, w, b, y = case(dtype=torch.float32)
    h.requires_grad_()
    s = torch.tensor(0.5, requires_grad=True)
    (d,) = torch.autograd.grad(s * rl.linear_cross_entropy_autograd(h, w, b, y), h, create_graph=True)
    (ds,) = torch.autograd.grad(d.sum(), s)
    assert torch.allclose(ds, ce_formula(h.detach(), w, b, y)[1].sum(), atol=1e-6)


@pytest.mark.gpu
def test_second_derivatives_are_refused_on_the_device():
    s = torch.randn(4, 9, device="cuda:0").log_softmax(-1).requires_grad_()
    loss = rl.reverse_kl_autograd(s, s.detach() - 0.1, torch.ones(4, 9, dtype=torch.bool, device="cuda:0"))
    (d,) = torch.autograd.grad(loss, s, create_graph=True)
    with pytest.raises(RuntimeError, match="reverse_kl_autograd.*first derivatives"):
        d.square().sum().backward()
    z = torch.randn(4, 300, device="cuda:0", requires_grad=True)
    loss = rl.reverse_kl_logits_autograd(z, z.detach().flip(0), torch.ones(4, dtype=torch.bool, device="cuda:0"))
    (d,) = torch.autograd.grad(loss, z, create_graph=True)
    with pytest.raises(RuntimeError, match="reverse_kl_logits_autograd.*first derivatives"):
        d.square().sum().backward()


def test_the_loss_alone_traces(on_cpu):
    """Where no input needs a gradient the loss is an op of its own, with a fake: it traces as the other forms do."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        h, w, y = torch.empty(4, 5, 16, dtype=torch.bfloat16), torch.empty(30, 16, dtype=torch.bfloat16), torch.empty(4, 5, dtype=torch.int64)
        loss = rl.linear_cross_entropy_autograd(h, w, None, y, z_loss=1e-3, reduction="sum")
        assert loss.shape == () and loss.dtype == torch.float32
        with torch.no_grad():
            assert rl.linear_cross_entropy_autograd(h.requires_grad_(), w, w[:, 0], y).shape == ()
    h, w, b, y = case()
    h.requires_grad_()
    want = ce_formula(h.detach(), w, b, y, z_loss=0.01)[0]
    compiled = torch.compile(lambda *a: 2 * rl.linear_cross_entropy_autograd(*a, z_loss=0.01), fullgraph=True, backend="aot_eager")
    with torch.no_grad():
        assert torch.equal(compiled(h, w, b, y), 2 * want)
    assert torch.equal(rl.linear_cross_entropy_autograd(h.detach(), w, b, y, z_loss=0.01), want)


@pytest.mark.gpu
def test_the_loss_alone_traces_on_the_device():
    h, w, b, y = (t.to("cuda:0") for t in case(70, 64, 300))
    compiled = torch.compile(lambda *a: rl.linear_cross_entropy_autograd(*a, z_loss=0.01), fullgraph=True, backend="aot_eager")
    want = rl.linear_cross_entropy_fwd(h, w, b, y, z_loss=0.01)
    assert torch.equal(compiled(h, w, b, y), want)
    w.requires_grad_()
    with torch.inference_mode():
        assert torch.equal(rl.linear_cross_entropy_autograd(h, w, b, y, z_loss=0.01), want)
    assert torch.equal(compiled(h, w, b, y).detach(), want)                  # and with a gradient


def test_forward_mode_tangents_are_refused(on_cpu):
    """An input that carries a tangent would lose it in the op: the result's derivative would be taken for zero."""
    import torch.autograd.forward_ad as forward
    h, w, b, y = case(dtype=torch.float32)
    ones = torch.ones(3, 4, dtype=torch.bool)
    lp = torch.randn(3, 4)
    forms = [(rl.linear_cross_entropy_autograd, [h, w, b, y], (0, 1, 2)),
             (rl.selective_logprob_autograd, [h, w, b, y], (0, 1, 2)),
             (rl.layer_norm_autograd, [h, w[0], b[:8]], (0, 1, 2)),
             (rl.reverse_kl_autograd, [lp, lp, ones], (0, 1)), (rl.reverse_kl_logits_autograd, [lp, lp, ones[:, 0]], (0, 1)),
             (rl.bnpo_loss_autograd, [lp, lp, None, lp[:, 0], ones], (0, 1, 3)),
             (rl.grpo_loss_autograd, [lp, lp, lp, lp[:, 0], ones], (0, 1, 2, 3))]
    for form, args, places in forms:
        for i in places:
            for needs in (False, True):
                with forward.dual_level():
                    dual = forward.make_dual(args[i].clone().requires_grad_(needs), torch.ones_like(args[i]))
                    with pytest.raises(RuntimeError, match="forward-mode"):
                        form(*args[:i], dual, *args[i + 1:])
    with forward.dual_level():
        assert torch.equal(rl.linear_cross_entropy_autograd(h, w, b, y), ce_formula(h, w, b, y)[0])
    with pytest.raises(RuntimeError, match="forward-mode"):
        torch.func.jvp(lambda t: rl.linear_cross_entropy_autograd(t, w, b, y), (h,), (h,))
