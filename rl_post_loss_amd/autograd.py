"""Autograd-aware entry points (model card "Geometric-AI Kernels", section
"Entry points": ``<name>_autograd``, the same kernel registered as a torch
custom op with an autograd formula, so that ``loss.backward()`` works and the
call traces under ``torch.compile(fullgraph=True)``).

Each op runs the fused forward+backward launch of the C ABI once, returns the
loss and keeps the gradient the launch wrote; backward multiplies that
gradient by the incoming scalar gradient of the loss (the chain rule for a
scalar loss), in float32, rounding once to the gradient's dtype.  There is no
other computation and no fallback: the ops call the same HIP kernels as the
direct entry points.  The gradient is an output of the op beside the loss; no
tensor is made for its own gradient, which a first backward pass does not ask
for.  It is a value, not a function of the inputs, so a second derivative raises,
and so does a forward-mode one.

The direct entry points stay the lowest-overhead path; these add the custom-op
dispatch (and, under compile, a graph break-free call).

A backward pass is captured into a graph only while no eager graph of the same
leaves lives: torch's gradient accumulators belong to the stream that made them,
and a capture that meets another stream's ends the process.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.forward_ad import unpack_dual

from . import _policy, _rkl, _rkl_logits, selective_logprob_bwd, selective_logprob_fwd
from .scoring import token_logprobs_bwd, token_logprobs_fwd
from .training import (layer_norm_bwd, layer_norm_fwd, linear_cross_entropy, linear_cross_entropy_fwd, rms_norm_bwd,
                       rms_norm_fwd)

__all__ = ["bnpo_loss_autograd", "grpo_loss_autograd", "reverse_kl_autograd",
           "reverse_kl_logits_autograd", "selective_logprob_autograd", "layer_norm_autograd",
           "linear_cross_entropy_autograd", "rms_norm_autograd", "token_logprobs_autograd"]

_LIB = "rlpl"


def _scaled(g: torch.Tensor, grad_loss: torch.Tensor) -> torch.Tensor:
    """g * grad_loss with the product formed in float32 and rounded once to g's dtype
    (grad_loss itself is never rounded to a half-precision type)."""
    return (g.float() * grad_loss.float()).to(g.dtype)


def _first_only(form: str, *grads) -> None:
    """Raises where a gradient arrives for an output that has no formula for it (a gradient's own, a statistic's)."""
    if any(g is not None for g in grads):
        raise RuntimeError(f"{form} gives first derivatives of its result only")


def _no_tangents(*inputs) -> None:
    """Raises where an input carries a forward-mode tangent: an op without a formula for it would drop it."""
    if any(t is not None and unpack_dual(t).tangent is not None for t in inputs):
        raise RuntimeError("the autograd forms have no forward-mode derivatives")


def _policy_op(op: str):
    @torch.library.custom_op(f"{_LIB}::{op}_loss", mutates_args=())
    def fused(policy_logprobs: torch.Tensor, old_policy_logprobs: torch.Tensor,
              ref_logprobs: Optional[torch.Tensor], advantages: torch.Tensor,
              completions_mask: torch.Tensor, epsilon: float, epsilon_high: float,
              beta: float, sign_aware: bool) -> Tuple[torch.Tensor, torch.Tensor]:
        loss, grad = _policy(op, True, policy_logprobs, old_policy_logprobs, ref_logprobs, advantages,
                             completions_mask, epsilon, epsilon_high, beta, False, None,
                             "sign_aware" if sign_aware else "literal")
        return loss, grad

    @fused.register_fake
    def _(policy_logprobs, old_policy_logprobs, ref_logprobs, advantages, completions_mask, epsilon,
          epsilon_high, beta, sign_aware):
        return (policy_logprobs.new_empty((), dtype=torch.float32), torch.empty_like(policy_logprobs))

    def setup_context(ctx, inputs, output):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(output[1])

    def backward(ctx, grad_loss, grad_of_grad):
        _first_only(f"{op}_loss_autograd", grad_of_grad)
        if grad_loss is None:
            return (None,) * 9
        (g,) = ctx.saved_tensors
        return (_scaled(g, grad_loss), None, None, None, None, None, None, None, None)

    fused.register_autograd(backward, setup_context=setup_context)
    return fused


def _rkl_op(name: str, direct):
    @torch.library.custom_op(f"{_LIB}::{name}", mutates_args=())
    def fused(student: torch.Tensor, teacher: torch.Tensor,
              completions_mask: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        loss, grad = direct(True, student, teacher, completions_mask, False, None)
        return loss, grad

    @fused.register_fake
    def _(student, teacher, completions_mask):
        return student.new_empty((), dtype=torch.float32), torch.empty_like(student)

    def setup_context(ctx, inputs, output):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(output[1])

    def backward(ctx, grad_loss, grad_of_grad):
        _first_only(f"{name}_autograd", grad_of_grad)
        if grad_loss is None:
            return None, None, None
        (g,) = ctx.saved_tensors
        return _scaled(g, grad_loss), None, None

    fused.register_autograd(backward, setup_context=setup_context)
    return fused


_bnpo = _policy_op("bnpo")
_grpo = _policy_op("grpo")
_rkl_tok = _rkl_op("reverse_kl", _rkl)
_rkl_vocab = _rkl_op("reverse_kl_logits", _rkl_logits)


def bnpo_loss_autograd(policy_logprobs, old_policy_logprobs, ref_logprobs, advantages, completions_mask, *,
                       epsilon=0.2, epsilon_high=None, beta=0.0, clip="literal"):
    """BNPO loss as a differentiable 0-d float32 tensor (gradient flows to policy_logprobs)."""
    _no_tangents(policy_logprobs, old_policy_logprobs, ref_logprobs, advantages)
    eh = epsilon if epsilon_high is None else epsilon_high
    return _bnpo(policy_logprobs, old_policy_logprobs, ref_logprobs, advantages, completions_mask,
                 float(epsilon), float(eh), float(beta), _sign_aware(clip))[0]


def grpo_loss_autograd(policy_logprobs, old_policy_logprobs, ref_logprobs, advantages, completions_mask, *,
                       epsilon=0.2, epsilon_high=None, beta=0.0, clip="literal"):
    """GRPO loss as a differentiable 0-d float32 tensor."""
    _no_tangents(policy_logprobs, old_policy_logprobs, ref_logprobs, advantages)
    eh = epsilon if epsilon_high is None else epsilon_high
    return _grpo(policy_logprobs, old_policy_logprobs, ref_logprobs, advantages, completions_mask,
                 float(epsilon), float(eh), float(beta), _sign_aware(clip))[0]


def _sign_aware(clip: str) -> bool:
    if clip not in ("literal", "sign_aware"):
        raise ValueError("clip must be 'literal' or 'sign_aware'")
    return clip == "sign_aware"


def reverse_kl_autograd(student_logprobs, teacher_logprobs, completions_mask):
    """Per-token reverse KL as a differentiable 0-d float32 tensor (gradient flows to the student)."""
    _no_tangents(student_logprobs, teacher_logprobs)
    return _rkl_tok(student_logprobs, teacher_logprobs, completions_mask)[0]


def reverse_kl_logits_autograd(student_logits, teacher_logits, completions_mask):
    """Full-vocab reverse KL as a differentiable 0-d float32 tensor (gradient flows to the student logits)."""
    _no_tangents(student_logits, teacher_logits)
    return _rkl_vocab(student_logits, teacher_logits, completions_mask)[0]


@torch.library.custom_op(f"{_LIB}::selective_logprob", mutates_args=())
def _selective(hidden: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
               targets: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    return selective_logprob_fwd(hidden, weight, bias, targets)


@_selective.register_fake
def _(hidden, weight, bias, targets):
    n = hidden.shape[0]
    return (hidden.new_empty((n,), dtype=torch.float32), hidden.new_empty((n,), dtype=torch.float32))


@torch.library.custom_op(f"{_LIB}::selective_logprob_backward", mutates_args=())
def _selective_bwd(hidden: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                   targets: torch.Tensor, lse: torch.Tensor, grad_logp: torch.Tensor,
                   need_hidden: bool, need_weight: bool) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    dh, dw, db = selective_logprob_bwd(hidden, weight, bias, targets, lse, grad_logp,
                                       need_hidden=need_hidden, need_weight=need_weight)
    # custom ops return tensors only: empty placeholders stand for the gradients not asked for
    empty = hidden.new_empty((0,))
    return (dh if dh is not None else empty, dw if dw is not None else empty.float(),
            db if db is not None else empty.float())


@_selective_bwd.register_fake
def _(hidden, weight, bias, targets, lse, grad_logp, need_hidden, need_weight):
    n, H = hidden.shape
    V = weight.shape[0]
    dh = hidden.new_empty((n, H)) if need_hidden else hidden.new_empty((0,))
    dw = hidden.new_empty((V, H), dtype=torch.float32) if need_weight else hidden.new_empty((0,), dtype=torch.float32)
    db = hidden.new_empty((V,) if bias is not None else (0,), dtype=torch.float32)
    return dh, dw, db


def _selective_setup(ctx, inputs, output):
    ctx.set_materialize_grads(False)
    hidden, weight, bias, targets = inputs
    ctx.has_bias = bias is not None
    ctx.save_for_backward(hidden, weight, bias, targets, output[1])


def _selective_backward(ctx, grad_logp, grad_lse):
    _first_only("selective_logprob_autograd", grad_lse)
    hidden, weight, bias, targets, lse = ctx.saved_tensors
    need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
    need_b = ctx.has_bias and ctx.needs_input_grad[2]
    if grad_logp is None or not (need_h or need_w or need_b):
        return None, None, None, None
    dh, dw, db = _selective_bwd(hidden, weight, bias, targets, lse, grad_logp, need_h, need_w)
    return (dh if need_h else None, dw.to(weight.dtype) if need_w else None,
            db.to(bias.dtype) if need_b else None, None)


_selective.register_autograd(_selective_backward, setup_context=_selective_setup)


def selective_logprob_autograd(hidden, weight, bias, targets):
    """Per-token target log-probabilities (float32, (n,)) as a differentiable tensor: gradients flow to
    hidden, weight and bias (the weight and bias gradients are formed in float32, then cast to their dtype)."""
    _no_tangents(hidden, weight, bias)
    return _selective(hidden, weight, bias, targets)[0]


@torch.library.custom_op(f"{_LIB}::layer_norm", mutates_args=())
def _norm(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
          eps: float) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return layer_norm_fwd(x, weight, bias, eps=eps)


@_norm.register_fake
def _(x, weight, bias, eps):
    stat = x.new_empty(x.shape[:-1], dtype=torch.float32)
    return x.new_empty(x.shape), stat, torch.empty_like(stat)


@torch.library.custom_op(f"{_LIB}::layer_norm_backward", mutates_args=())
def _norm_bwd(grad_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
              rstd: torch.Tensor, need_x: bool, need_weight: bool, need_bias: bool,
              bias_dtype: Optional[torch.dtype] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    out = layer_norm_bwd(grad_y, x, weight, mean, rstd, need_x=need_x, need_weight=need_weight, need_bias=need_bias,
                         bias_dtype=bias_dtype)
    return tuple(x.new_empty((0,)) if t is None else t for t in out)


@_norm_bwd.register_fake
def _(grad_y, x, weight, mean, rstd, need_x, need_weight, need_bias, bias_dtype=None):
    vec = x.new_empty(x.shape[-1:], dtype=weight.dtype if weight is not None else bias_dtype or x.dtype)
    none = x.new_empty((0,))
    return (x.new_empty(x.shape) if need_x else none, vec if need_weight and weight is not None else none.clone(),
            torch.empty_like(vec) if need_bias else none.clone())


def _norm_setup(ctx, inputs, output):
    x, weight, bias, _ = inputs
    ctx.set_materialize_grads(False)
    ctx.bias_dtype = None if bias is None else bias.dtype
    ctx.save_for_backward(x, weight, output[1], output[2])


def _norm_backward(ctx, grad_y, grad_mean, grad_rstd):
    _first_only("layer_norm_autograd", grad_mean, grad_rstd)
    x, weight, mean, rstd = ctx.saved_tensors
    need_x, need_w = ctx.needs_input_grad[0], weight is not None and ctx.needs_input_grad[1]
    need_b = ctx.bias_dtype is not None and ctx.needs_input_grad[2]
    if grad_y is None or not (need_x or need_w or need_b):
        return None, None, None, None
    dx, dw, db = _norm_bwd(grad_y, x, weight, mean, rstd, need_x, need_w, need_b, ctx.bias_dtype)
    return dx if need_x else None, dw if need_w else None, db if need_b else None, None


_norm.register_autograd(_norm_backward, setup_context=_norm_setup)


def layer_norm_autograd(x, weight=None, bias=None, *, eps=1e-5):
    """Layer norm over the last dimension as a differentiable tensor of x's shape and dtype (gradients flow to x,
    weight and bias; the saved statistics are float32)."""
    _no_tangents(x, weight, bias)
    return _norm(x, weight, bias, float(eps))[0]


@torch.library.custom_op(f"{_LIB}::rms_norm", mutates_args=())
def _rms(x: torch.Tensor, weight: Optional[torch.Tensor], residual: Optional[torch.Tensor],
         eps: float) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    y, rstd, h = rms_norm_fwd(x, weight, residual, eps=eps)
    return y, rstd, x.new_empty((0,)) if h is None else h


@_rms.register_fake
def _(x, weight, residual, eps):
    return (x.new_empty(x.shape), x.new_empty(x.shape[:-1], dtype=torch.float32),
            x.new_empty((0,)) if residual is None else residual.new_empty(residual.shape))


@torch.library.custom_op(f"{_LIB}::rms_norm_backward", mutates_args=())
def _rms_bwd(grad_y: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
             grad_stream: Optional[torch.Tensor], need_h: bool, need_weight: bool) -> Tuple[torch.Tensor, torch.Tensor]:
    out = rms_norm_bwd(grad_y, h, weight, rstd, grad_stream, need_h=need_h, need_weight=need_weight)
    return tuple(h.new_empty((0,)) if t is None else t for t in out)


@_rms_bwd.register_fake
def _(grad_y, h, weight, rstd, grad_stream, need_h, need_weight):
    return (h.new_empty(h.shape) if need_h else h.new_empty((0,)),
            weight.new_empty(weight.shape) if need_weight and weight is not None else h.new_empty((0,)))


def _rms_setup(ctx, inputs, output):
    x, weight, residual, _ = inputs
    ctx.set_materialize_grads(False)
    ctx.dtypes = x.dtype, None if residual is None else residual.dtype
    ctx.save_for_backward(x if residual is None else output[2], weight, output[1])


def _rms_backward(ctx, grad_y, grad_rstd, grad_h):
    _first_only("rms_norm_autograd", grad_rstd)
    h, weight, rstd = ctx.saved_tensors
    x_dtype, r_dtype = ctx.dtypes
    need_x, need_w, need_r = ctx.needs_input_grad[0], weight is not None and ctx.needs_input_grad[1], ctx.needs_input_grad[2]
    if r_dtype is None:
        grad_h = None
    dh = grad_h
    dw = None
    if grad_y is not None and (need_x or need_r or need_w):
        dh, dw = _rms_bwd(grad_y, h, weight, rstd, grad_h, need_x or need_r, need_w)
    elif dh is None:
        return None, None, None, None
    return dh.to(x_dtype) if need_x else None, dw if need_w else None, dh.to(r_dtype) if need_r else None, None


_rms.register_autograd(_rms_backward, setup_context=_rms_setup)


def rms_norm_autograd(x, weight=None, residual=None, *, eps=1e-6):
    """RMS norm over the last dimension as a differentiable tensor of x's shape and dtype, or with a residual (y, h), h =
    x + residual in the residual's dtype.  Gradients flow to x, weight and residual."""
    _no_tangents(x, weight, residual)
    y, _, h = _rms(x, weight, residual, float(eps))
    return y if residual is None else (y, h)


@torch.library.custom_op(f"{_LIB}::token_logprobs", mutates_args=())
def _token(logits: torch.Tensor, targets: torch.Tensor, mask: Optional[torch.Tensor],
           temperature: float) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    logp, lse, entropy, _, _ = token_logprobs_fwd(logits, targets, mask, temperature=temperature)
    return logp, entropy, lse


@_token.register_fake
def _(logits, targets, mask, temperature):
    out = logits.new_empty(logits.shape[:-1], dtype=torch.float32)
    return out, torch.empty_like(out), torch.empty_like(out)


@torch.library.custom_op(f"{_LIB}::token_logprobs_backward", mutates_args=())
def _token_bwd(logits: torch.Tensor, targets: torch.Tensor, mask: Optional[torch.Tensor], lse: torch.Tensor,
               entropy: torch.Tensor, grad_logp: Optional[torch.Tensor], grad_entropy: Optional[torch.Tensor],
               temperature: float) -> torch.Tensor:
    return token_logprobs_bwd(logits, targets, mask, lse, entropy, grad_logp, grad_entropy, temperature=temperature)


@_token_bwd.register_fake
def _(logits, targets, mask, lse, entropy, grad_logp, grad_entropy, temperature):
    return logits.new_empty(logits.shape)


def _token_setup(ctx, inputs, output):
    logits, targets, mask, temperature = inputs
    ctx.set_materialize_grads(False)
    ctx.temperature = temperature
    ctx.save_for_backward(logits, targets, mask, output[2], output[1])


def _token_backward(ctx, grad_logp, grad_entropy, grad_lse):
    _first_only("token_logprobs_autograd", grad_lse)
    if (grad_logp is None and grad_entropy is None) or not ctx.needs_input_grad[0]:
        return None, None, None, None
    logits, targets, mask, lse, entropy = ctx.saved_tensors
    return _token_bwd(logits, targets, mask, lse, entropy, grad_logp, grad_entropy, ctx.temperature), None, None, None


_token.register_autograd(_token_backward, setup_context=_token_setup)


def token_logprobs_autograd(logits, targets, mask=None, *, temperature=1.0):
    """(logp, entropy) of ``token_logprobs_fwd`` as differentiable float32 tensors of the logits' leading shape: gradients
    of both flow to the logits, in one pass that writes them."""
    _no_tangents(logits)
    return _token(logits, targets, mask, float(temperature))[:2]


def _ce_held(dtype: torch.dtype) -> torch.dtype:
    """What the gradients are held in between the two passes.  A mean's 1 / N takes many of them below fp16's normal
    range, and the incoming gradient, which may be a loss scale against that, comes later: they stay in float32."""
    return torch.float32 if dtype == torch.float16 else dtype


@torch.library.custom_op(f"{_LIB}::linear_cross_entropy", mutates_args=())
def _ce(hidden: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], targets: torch.Tensor,
        ignore_index: int, z_loss: float, reduction: str, need_hidden: bool, need_weight: bool,
        need_bias: bool) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    held = _ce_held(hidden.dtype)
    loss, *grads = linear_cross_entropy(hidden, weight, bias, targets, ignore_index=ignore_index, z_loss=z_loss,
                                        reduction=reduction, need_hidden=need_hidden, need_weight=need_weight,
                                        need_bias=need_bias, weight_grad_dtype=held, hidden_grad_dtype=held)
    return (loss, *(hidden.new_empty((0,)) if g is None else g for g in grads))


@_ce.register_fake
def _(hidden, weight, bias, targets, ignore_index, z_loss, reduction, need_hidden, need_weight, need_bias):
    held = _ce_held(hidden.dtype)
    none = lambda: hidden.new_empty((0,))  # noqa: E731
    return (hidden.new_empty((), dtype=torch.float32), hidden.new_empty(hidden.shape, dtype=held) if need_hidden else none(),
            weight.new_empty(weight.shape, dtype=held) if need_weight else none(),
            bias.new_empty(bias.shape, dtype=held) if need_bias and bias is not None else none())


def _ce_setup(ctx, inputs, output):
    ctx.set_materialize_grads(False)
    ctx.save_for_backward(*output[1:])
    ctx.dtype = inputs[0].dtype
    ctx.need = inputs[7:9] + (inputs[9] and inputs[2] is not None,)


def _scaled_once(g, grad_loss, dtype):
    """_scaled to dtype in one pass, without float32 tensors of g's size (128256 x 4096 bf16: 462 us instead of 1758)."""
    if torch.is_grad_enabled():            # the formula's own gradient is wanted
        return _scaled(g, grad_loss).to(dtype)
    return torch.mul(g, grad_loss.float().view(1), out=torch.empty_like(g, dtype=dtype))


def _ce_backward(ctx, grad_loss, *grads_of_grads):
    _first_only("linear_cross_entropy_autograd", *grads_of_grads)
    if grad_loss is None:
        return (None,) * 10
    grads = [_scaled_once(g, grad_loss, ctx.dtype) if need else None for g, need in zip(ctx.saved_tensors, ctx.need)]
    return (*grads, None, None, None, None, None, None, None)


_ce.register_autograd(_ce_backward, setup_context=_ce_setup)


@torch.library.custom_op(f"{_LIB}::linear_cross_entropy_loss", mutates_args=())
def _ce_loss(hidden: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], targets: torch.Tensor,
             ignore_index: int, z_loss: float, reduction: str) -> torch.Tensor:
    return linear_cross_entropy_fwd(hidden, weight, bias, targets, ignore_index=ignore_index, z_loss=z_loss,
                                    reduction=reduction)


@_ce_loss.register_fake
def _(hidden, weight, bias, targets, ignore_index, z_loss, reduction):
    return hidden.new_empty((), dtype=torch.float32)


def linear_cross_entropy_autograd(hidden, weight, bias, targets, *, ignore_index=-100, z_loss=0.0, reduction="mean"):
    """The loss of ``linear_cross_entropy`` as a differentiable 0-d float32 tensor: gradients flow to hidden, weight and
    bias.  They are formed with the loss, for the inputs that need one (fp16 ones are held in float32 until the incoming
    gradient, a loss scale for instance, has been applied); where none does, the loss alone is."""
    _no_tangents(hidden, weight, bias)
    needs = [t is not None and t.requires_grad and torch.is_grad_enabled() for t in (hidden, weight, bias)]
    if not any(needs):
        return _ce_loss(hidden, weight, bias, targets, int(ignore_index), float(z_loss), reduction)
    return _ce(hidden, weight, bias, targets, int(ignore_index), float(z_loss), reduction, *needs)[0]
