"""Operators of a training step around the losses, over the same C ABI.

* ``linear_cross_entropy`` / ``linear_cross_entropy_fwd``: the softmax cross entropy of an output projection over a
  large vocabulary, with the gradients of the hidden states, the projection and its bias;
* ``layer_norm_fwd`` / ``layer_norm_bwd``: the norm of the hidden states that the output projection reads,
  with the reduction of its weight's and bias's gradients;
* ``rms_norm_fwd`` / ``rms_norm_fp8`` / ``rms_norm_bwd``: the norm by the root mean square, with the residual's addition,
  in the input's type or in 8 bits with scales;
* ``adamw_plan`` / ``adamw_step``: one AdamW step over a list of tensors, moments in float32 or in 8 bits;
* ``grad_norm`` / ``scale_grads`` / ``clip_grads``: the norm over a list of gradients, and clipping.

As in the package's other entry points, this module marshals arguments only: every step runs in the library's HIP
kernels on the current stream of the tensors' device, without synchronising.
"""
from __future__ import annotations

import ctypes
import math
from array import array
from contextlib import nullcontext
from typing import Optional, Sequence

import numpy as np
import torch

from torch.autograd.graph import increment_version

from . import DTYPE, _aligned, _check, _ws_ptr, library

__all__ = ["linear_cross_entropy", "linear_cross_entropy_fwd", "layer_norm_fwd", "layer_norm_bwd", "adamw_plan", "adamw_step", "AdamWPlan",
           "rms_norm_fwd", "rms_norm_fp8", "rms_norm_bwd", "grad_norm", "scale_grads", "clip_grads"]

REDUCTION = {"mean": 0, "sum": 1}
CE_HIDDEN_F32 = 1    # rlpl_linear_cross_entropy flags (RLPL_CE_HIDDEN_F32)

BLOCK = 256   # values of an 8-bit moment that share one scale


_HERE = nullcontext()


def _on(device: torch.device):
    """The device as the current one: the library launches on the current device."""
    return _HERE if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def _stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)   # the current stream's handle, without a Stream object


def _dense(t: torch.Tensor) -> torch.Tensor:
    t = t if t.is_contiguous() else t.contiguous()
    return t.detach() if t.requires_grad else t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _empty(shape, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """torch.empty, which takes sizes one by one 0.4 us faster than a tuple of them."""
    return torch.empty(*shape, dtype=dtype, device=device) if shape else torch.empty((), dtype=dtype, device=device)


def _scratch(nbytes: int, workspace: Optional[torch.Tensor], device: torch.device, fn: str) -> torch.Tensor:
    if nbytes == 0:
        _check(fn, 2)
    if workspace is None:
        return torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    if workspace.device != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace


# ------------------------------------------------------------------------------------- vocabulary cross entropy

def _plain(t: torch.Tensor) -> torch.Tensor:
    return t.detach() if t.requires_grad else t


def _ce_operands(hidden, weight, bias, targets, reduction):
    for name, t in (("hidden", hidden), ("weight", weight)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    x, w, b, y = _plain(hidden), _plain(weight), None, targets
    dt, dev, shape, wshape = x.dtype, x.device, x.shape, w.shape
    if dt not in (torch.float16, torch.bfloat16) or w.dtype != dt:
        raise TypeError("hidden and weight must share a float16 or bfloat16 dtype")
    if len(shape) < 1 or len(wshape) != 2 or shape[-1] != wshape[1] or w.device != dev:
        raise ValueError("hidden (*, H) and weight (V, H) must agree in H and device")
    if bias is not None:
        b = _plain(bias)
        if b.dtype != dt or b.dim() != 1 or b.shape[0] != wshape[0] or b.device != dev:
            raise ValueError(f"bias must be a ({wshape[0]},) tensor of the operands' dtype and device")
        b = b.contiguous()
    if y.dtype != torch.int64 or y.shape != shape[:-1] or y.device != dev:
        raise ValueError(f"targets must be an int64 {tuple(shape[:-1])} tensor on the operands' device")
    if reduction not in REDUCTION:
        raise ValueError(f"reduction must be one of {sorted(REDUCTION)}")
    if x.numel() == 0 or w.numel() == 0:
        _check("linear_cross_entropy", 2)
    x, y = _aligned(x), y.contiguous()
    if len(shape) != 2:
        x, y = x.view(-1, shape[-1]), y.view(-1)
    return x, _aligned(w), b, y


def linear_cross_entropy_fwd(hidden, weight, bias, targets, *, ignore_index=-100, z_loss=0.0, reduction="mean",
                             workspace=None):
    """The loss of ``linear_cross_entropy`` (a 0-d float32 tensor, bit-identical), without gradients."""
    x, w, b, y = _ce_operands(hidden, weight, bias, targets, reduction)
    (n, H), V, dev, lib = x.shape, w.shape[0], x.device, library()
    ws = _scratch(lib.linear_cross_entropy_workspace_bytes(n, H, V, 0), workspace, dev,
                  "linear_cross_entropy_workspace_bytes")
    wp, wn = _ws_ptr(ws)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    with _on(dev):
        _check("linear_cross_entropy_fwd", lib.linear_cross_entropy_fwd(
            x.data_ptr(), w.data_ptr(), _ptr(b), y.data_ptr(), n, H, V, DTYPE[x.dtype], int(ignore_index), float(z_loss),
            REDUCTION[reduction], loss.data_ptr(), wp, wn, _stream(dev)))
    return loss


def linear_cross_entropy(hidden, weight, bias, targets, *, ignore_index=-100, z_loss=0.0, reduction="mean",
                         need_hidden=True, need_weight=True, need_bias=True, weight_grad_dtype=None, grad_weight=None,
                         grad_bias=None, workspace=None, hidden_grad_dtype=None):
    """Softmax cross entropy of the logits hidden . weight^T + bias, with its gradients, in pieces of the vocabulary:
    (loss, grad_hidden, grad_weight, grad_bias), None for gradients not wanted and for a bias that is not there (unless
    its gradient is passed to be added to).  Up to 2^27 logits are held in float32 (all of 1024 x 128256, in a
    workspace of 0.93 GB), the others are formed twice.

    hidden (*, H) and weight (V, H) float16 or bfloat16, H a multiple of 8; bias (V,) or None; targets int64, of hidden's
    leading shape.  Rows whose target is ``ignore_index`` do not count.  loss is the mean (or sum) over the others of
    lse - z[target] + z_loss * lse^2, a 0-d float32 tensor, and 0 where no row counts.  0 <= z_loss <= 1; with fp16 operands
    the penalty's factor 1 + 2 z_loss lse fits where |lse| <= 500 (beyond, gradients may overflow to NaN).

    weight_grad_dtype: the operands' dtype (the default) or torch.float32, of grad_weight and grad_bias;
    hidden_grad_dtype: likewise, of grad_hidden.  Passing ``grad_weight`` / ``grad_bias`` (contiguous float32) adds to
    them, over groups of tokens or micro-batches."""
    x, w, b, y = _ce_operands(hidden, weight, bias, targets, reduction)
    (n, H), V, dev, lib = x.shape, w.shape[0], x.device, library()
    need_bias = need_bias and (b is not None or grad_bias is not None)
    accumulate = grad_weight is not None or grad_bias is not None
    if accumulate:
        if weight_grad_dtype not in (None, torch.float32):
            raise ValueError("gradients are added to in float32")
        weight_grad_dtype = torch.float32
        if (need_weight and grad_weight is None) or (need_bias and grad_bias is None):
            raise ValueError("to accumulate, pass both grad_weight (when wanted) and grad_bias (with a bias)")
    wdt = x.dtype if weight_grad_dtype is None else weight_grad_dtype
    if wdt not in (x.dtype, torch.float32):
        raise TypeError("weight_grad_dtype must be the operands' dtype or float32")
    if hidden_grad_dtype not in (None, x.dtype, torch.float32):
        raise TypeError("hidden_grad_dtype must be the operands' dtype or float32")
    wide = hidden_grad_dtype is torch.float32
    for name, t, shape in (("grad_weight", grad_weight, (V, H)), ("grad_bias", grad_bias, (V,))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous()
                              or t.device != dev):
            raise ValueError(f"{name} must be a contiguous float32 {shape} tensor on the operands' device")
    dh = torch.empty_like(x, dtype=hidden_grad_dtype) if need_hidden else None
    dw = (grad_weight if accumulate else torch.empty((V, H), dtype=wdt, device=dev)) if need_weight else None
    db = (grad_bias if accumulate else torch.empty(V, dtype=wdt, device=dev)) if need_bias else None
    ws = _scratch(lib.linear_cross_entropy_workspace_bytes(n, H, V, 1), workspace, dev,
                  "linear_cross_entropy_workspace_bytes")
    wp, wn = _ws_ptr(ws)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    args = (x.data_ptr(), w.data_ptr(), _ptr(b), y.data_ptr(), n, H, V, DTYPE[x.dtype], int(ignore_index), float(z_loss),
            REDUCTION[reduction], loss.data_ptr(), _ptr(dh), _ptr(dw), _ptr(db), DTYPE[wdt], int(accumulate), wp, wn,
            _stream(dev))
    with _on(dev):
        _check("linear_cross_entropy",
               lib.rlpl_linear_cross_entropy(CE_HIDDEN_F32, *args) if wide else lib.linear_cross_entropy(*args))
    if accumulate:
        increment_version([t for t in (dw, db) if t is not None])   # a graph that saved an old value says so
    return loss, dh if dh is None or hidden.dim() == 2 else dh.view(hidden.shape), dw, db


# ------------------------------------------------------------------------------------------------------- layer norm

def _norm_rows(x: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() < 1:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor with at least one dimension")
    if x.dtype not in DTYPE:
        raise TypeError(f"{name} must be float32, float16 or bfloat16")
    if x.numel() == 0:
        _check("layer_norm", 2)
    return _dense(x)


def _norm_vector(v: Optional[torch.Tensor], name: str, x: torch.Tensor) -> Optional[torch.Tensor]:
    if v is None:
        return None
    if not isinstance(v, torch.Tensor) or v.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"{name} must be a tensor of the input's dtype or float32")
    if v.dim() != 1 or v.shape[0] != x.shape[-1] or v.device != x.device:
        raise ValueError(f"{name} must have shape ({x.shape[-1]},) on the input's device")
    return _dense(v)


def layer_norm_fwd(x, weight=None, bias=None, *, eps=1e-5):
    """Layer norm over the last dimension: (y, mean, rstd).  x (*, H) float32, float16 or bfloat16; weight and bias
    (H,) of x's dtype or both float32, or None (ones / zeros).  y has x's shape and dtype; mean and rstd are float32
    of x's leading shape, what the backward pass takes."""
    x = _norm_rows(x, "x")
    w, b = _norm_vector(weight, "weight", x), _norm_vector(bias, "bias", x)
    if w is not None and b is not None and w.dtype != b.dtype:
        raise TypeError("weight and bias must share a dtype")
    H = x.shape[-1]
    rows = x.numel() // H
    y = torch.empty_like(x)
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    wt = w if w is not None else b
    with _on(x.device):
        _check("layer_norm_fwd", library().layer_norm_fwd(
            x.data_ptr(), _ptr(w), _ptr(b), rows, H, DTYPE[x.dtype], DTYPE[x.dtype if wt is None else wt.dtype],
            float(eps), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _stream(x.device)))
    return y, mean, rstd


def layer_norm_bwd(grad_y, x, weight, mean, rstd, *, need_x=True, need_weight=True, need_bias=True, workspace=None,
                   bias_dtype=None):
    """Gradients of sum(grad_y * y): (grad_x, grad_weight, grad_bias), None where not wanted.  mean and rstd are the
    forward's.  grad_x has x's dtype, the other two the weight's (float32 sums over the rows, rounded once).  Without a
    weight there is no grad_weight, and grad_bias has ``bias_dtype``: x's dtype (the default) or torch.float32, the
    bias's own; with one, bias_dtype is the weight's if it is given."""
    x = _norm_rows(x, "x")
    w = _norm_vector(weight, "weight", x)
    gy = _norm_rows(grad_y, "grad_y")
    if gy.shape != x.shape or gy.dtype != x.dtype or gy.device != x.device:
        raise ValueError("grad_y must match x in shape, dtype and device")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.shape != x.shape[:-1] or t.device != x.device:
            raise ValueError(f"{name} must be the forward's float32 tensor of shape {tuple(x.shape[:-1])}")
    mean, rstd = _dense(mean), _dense(rstd)
    H = x.shape[-1]
    rows = x.numel() // H
    wdt = w.dtype if w is not None else x.dtype if bias_dtype is None else bias_dtype
    if wdt not in (x.dtype, torch.float32) or bias_dtype not in (None, wdt):
        raise TypeError("bias_dtype must be the weight's dtype, or without a weight the input's or float32")
    dx = torch.empty_like(x) if need_x else None
    dw = torch.empty_like(w) if need_weight and w is not None else None
    db = (x.new_empty(H, dtype=wdt) if w is None else torch.empty_like(w)) if need_bias else None
    lib = library()
    ws = _scratch(lib.layer_norm_workspace_bytes(rows, H), workspace, x.device, "layer_norm_workspace_bytes")
    wp, wn = _ws_ptr(ws)
    with _on(x.device):
        _check("layer_norm_bwd", lib.layer_norm_bwd(
            gy.data_ptr(), x.data_ptr(), _ptr(w), mean.data_ptr(), rstd.data_ptr(), rows, H, DTYPE[x.dtype], DTYPE[wdt],
            _ptr(dx), _ptr(dw), _ptr(db), wp, wn, _stream(x.device)))
    return dx, dw, db


# ------------------------------------------------------------------------------------------------------- RMS norm

GROUP = 128   # columns of an 8-bit row that share one scale


def _rms_operands(x, weight, residual):
    x = _norm_rows(x, "x")
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in (x.dtype, torch.float32):
            raise TypeError("residual must be a tensor of x's dtype or float32")
        if residual.shape != x.shape or residual.device != x.device:
            raise ValueError("residual must match x in shape and device")
        residual = _dense(residual)
    return x, _norm_vector(weight, "weight", x), residual


def _rms_call(fn, x, w, residual, eps, outputs):
    *lead, H = x.shape
    dev, code = x.device, DTYPE[x.dtype]
    stream = None if residual is None else torch.empty_like(residual)
    rstd = _empty(lead, torch.float32, dev)
    with _on(dev):
        _check(fn, getattr(library(), fn)(
            x.data_ptr(), _ptr(w), _ptr(residual), x.numel() // H, H, code, code if w is None else DTYPE[w.dtype],
            code if residual is None else DTYPE[residual.dtype], float(eps), *[t.data_ptr() for t in outputs],
            rstd.data_ptr(), _ptr(stream), _stream(dev)))
    return rstd, stream


def rms_norm_fwd(x, weight=None, residual=None, *, eps=1e-6):
    """RMS norm over the last dimension of h = x + residual (x itself without a residual): (y, rstd, h), None for the
    last without a residual.

    x (*, H) float32, float16 or bfloat16, H up to 16384; weight (H,) of x's dtype or float32, or None (ones); residual of
    x's shape, of its dtype or float32.  y = h / sqrt(avg h^2 + eps) * weight has x's dtype; h, the new residual stream,
    has the residual's, and the norm is that of h as it is stored; rstd is float32 of x's leading shape."""
    x, w, residual = _rms_operands(x, weight, residual)
    y = torch.empty_like(x)
    return y, *_rms_call("rms_norm_fwd", x, w, residual, eps, (y,))


def rms_norm_fp8(x, weight=None, residual=None, *, eps=1e-6):
    """``rms_norm_fwd`` with y in 8 bits: (q, scale, rstd, h).  q has x's shape and dtype float8_e4m3fn; scale is float32
    (*, ceil(H / 128)), one for every 128 columns: y is about q * scale, as ``fp8_linear`` takes it."""
    x, w, residual = _rms_operands(x, weight, residual)
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    *lead, H = x.shape
    scale = _empty((*lead, (H + GROUP - 1) // GROUP), torch.float32, x.device)
    return q, scale, *_rms_call("rms_norm_fp8", x, w, residual, eps, (q, scale))


def rms_norm_bwd(grad_y, h, weight, rstd, grad_stream=None, *, need_h=True, need_weight=True, workspace=None):
    """Gradients of sum(grad_y * y) + sum(grad_stream * h): (grad_h, grad_weight), None where not wanted.  h and rstd are
    the forward's (h is x without a residual).  grad_h, the gradient of x and of the residual alike, has h's dtype;
    grad_weight the weight's (float32 sums over the rows, rounded once)."""
    gy = _norm_rows(grad_y, "grad_y")
    h = _norm_rows(h, "h")
    if h.shape != gy.shape or h.device != gy.device or h.dtype not in (gy.dtype, torch.float32):
        raise ValueError("h must match grad_y in shape and device, and have its dtype or float32")
    w = _norm_vector(weight, "weight", gy)
    if not isinstance(rstd, torch.Tensor) or rstd.dtype != torch.float32 or rstd.shape != h.shape[:-1] or rstd.device != h.device:
        raise ValueError(f"rstd must be the forward's float32 tensor of shape {tuple(h.shape[:-1])}")
    if grad_stream is not None:
        if not isinstance(grad_stream, torch.Tensor) or grad_stream.dtype != h.dtype or grad_stream.shape != h.shape \
                or grad_stream.device != h.device:
            raise ValueError("grad_stream must match h in shape, dtype and device")
        grad_stream = _dense(grad_stream)
    rstd, H = _dense(rstd), h.shape[-1]
    rows = h.numel() // H
    dh = torch.empty_like(h) if need_h else None
    dw = torch.empty_like(w) if need_weight and w is not None else None
    lib = library()
    ws = _scratch(lib.rms_norm_workspace_bytes(rows, H), workspace, h.device, "rms_norm_workspace_bytes")
    wp, wn = _ws_ptr(ws)
    with _on(h.device):
        _check("rms_norm_bwd", lib.rms_norm_bwd(
            gy.data_ptr(), h.data_ptr(), _ptr(w), rstd.data_ptr(), _ptr(grad_stream), rows, H, DTYPE[gy.dtype],
            DTYPE[gy.dtype if w is None else w.dtype], DTYPE[h.dtype], _ptr(dh), _ptr(dw), wp, wn, _stream(h.device)))
    return dh, dw


# ------------------------------------------------------------------------------------------------------- AdamW

def _pointers(tensors) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() if t is not None and t.numel() else None for t in tensors])


class AdamWPlan:
    """What stays the same between the steps over a list of tensors (see ``adamw_plan``): the parameters, their
    moments, copies and weight decays.

    ``params``, ``copies`` and the moments (``exp_avg``, ``exp_avg_sq``, and with 8-bit states ``exp_avg_scale``,
    ``exp_avg_sq_scale``) are lists of tensors that share storage with those given or made, so the plan keeps the
    memory it updates alive.  A parameter whose storage is replaced (``p.data = ...``) needs a new plan.  A plan may be
    dropped right after a step is enqueued, on any stream; a captured step needs its plan until the last replay."""

    def __init__(self, params, copies, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, weight_decay, made=()):
        self.params, self.copies = params, copies
        self.exp_avg, self.exp_avg_sq = exp_avg, exp_avg_sq
        self.exp_avg_scale, self.exp_avg_sq_scale = exp_avg_scale, exp_avg_sq_scale
        self.weight_decay = weight_decay
        self.device = params[0].device
        self.sizes = [p.numel() for p in params]
        self._shapes = [p.shape for p in params]
        count = len(params)
        sizes = (ctypes.c_int64 * count)(*self.sizes)
        lib = library()
        nbytes = lib.rlpl_adamw_plan_bytes(sizes, count)
        if nbytes == 0:
            _check("rlpl_adamw_plan_bytes", 2)
        self._host = np.zeros((nbytes + 7) // 8, dtype=np.uint64)
        eight = exp_avg_scale is not None
        _check("rlpl_adamw_plan_build", lib.rlpl_adamw_plan_build(
            self._host.ctypes.data, nbytes, sizes, count, _pointers(params), DTYPE[params[0].dtype],
            _pointers(copies) if copies is not None else None, DTYPE[copies[0].dtype] if copies is not None else 0,
            _pointers(exp_avg), _pointers(exp_avg_sq), _pointers(exp_avg_scale) if eight else None,
            _pointers(exp_avg_sq_scale) if eight else None, 8 if eight else 32,
            (ctypes.c_double * count)(*weight_decay)))
        self._device = torch.from_numpy(self._host.view(np.int64)).to(self.device)
        self._made = [self._device, *made]       # allocated here, on the current stream
        self._streams = {_stream(self.device)}   # streams that the allocator knows to use them

    def _used_on_current_stream(self, stream: int) -> None:
        """Tells the allocator, once a stream, that a plan dropped right after a step is still in use there."""
        for t in self._made:
            t.record_stream(torch.cuda.current_stream(self.device))
        self._streams.add(stream)

    def moments(self, i: int):
        """The first and second moment of tensor i in float32, in its shape (8-bit states as the values they stand for)."""
        shape = self.params[i].shape
        if self.exp_avg_scale is None:
            return self.exp_avg[i].view(shape), self.exp_avg_sq[i].view(shape)
        n = self.sizes[i]
        wide = lambda q, s: (q.view(-1).float() * s.repeat_interleave(BLOCK)[:n]).view(shape)  # noqa: E731
        return wide(self.exp_avg[i], self.exp_avg_scale[i]), wide(self.exp_avg_sq[i], self.exp_avg_sq_scale[i]).square()


def _alias(t, name, dtypes, device, numel=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (device is not None and t.device != device):
        raise TypeError(f"{name} must be CUDA (HIP) tensors on one device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous() or (numel is not None and t.numel() != numel):
        raise ValueError(f"{name} must be contiguous tensors" + ("" if numel is None else f" of {numel} elements here"))
    return t.detach()


def adamw_plan(params: Sequence[torch.Tensor], *, state_dtype=torch.float32, weight_decay=0.01, copies=None,
               exp_avg=None, exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None) -> AdamWPlan:
    """A plan of AdamW steps over ``params`` (contiguous, of one device and dtype: float32, float16 or bfloat16).

    state_dtype: torch.float32, or torch.float8_e4m3fn for moments in 8 bits (one float32 scale per 256 consecutive
    elements; ``exp_avg_sq`` then holds the second moment's root, which is right on average, and so its square a little
    high: 5 % with Gaussian gradients and beta2 = 0.999, an eighth at most in the normal range).  The moments are made,
    filled with zeros, unless they are given (``exp_avg``, ``exp_avg_sq``, and the scales with 8-bit ones), as when a
    run is resumed.
    weight_decay: a number, or one per tensor.  copies: float16 or bfloat16 tensors, one per float32 parameter, that
    every step writes with the new values."""
    params = list(params)
    if not params:
        raise ValueError("params is empty")
    dt = params[0].dtype if isinstance(params[0], torch.Tensor) else None
    dev = params[0].device if isinstance(params[0], torch.Tensor) else None
    if dt not in DTYPE:
        raise TypeError("params must be float32, float16 or bfloat16 tensors of one dtype")
    params = [_alias(p, "params", (dt,), dev) for p in params]
    sizes = [p.numel() for p in params]
    if copies is not None:
        copies = list(copies)
        if dt != torch.float32 or len(copies) != len(params):
            raise ValueError("copies are taken for float32 params, one each")
        cdt = copies[0].dtype
        if cdt not in (torch.float16, torch.bfloat16):
            raise TypeError("copies must be float16 or bfloat16")
        copies = [_alias(c, "copies", (cdt,), dev, n) for c, n in zip(copies, sizes)]
    given = exp_avg is not None
    if given != (exp_avg_sq is not None):
        raise ValueError("exp_avg and exp_avg_sq are given together")
    if given:
        exp_avg, exp_avg_sq = list(exp_avg), list(exp_avg_sq)
        if len(exp_avg) != len(params) or len(exp_avg_sq) != len(params):
            raise ValueError("exp_avg and exp_avg_sq need one tensor per parameter")
        state_dtype, made = exp_avg[0].dtype, []
    if state_dtype not in (torch.float32, torch.float8_e4m3fn):
        raise TypeError("moments must be float32 or float8_e4m3fn")
    eight = state_dtype == torch.float8_e4m3fn
    blocks = [(n + BLOCK - 1) // BLOCK for n in sizes]
    if given:
        exp_avg = [_alias(t, "exp_avg", (state_dtype,), dev, n) for t, n in zip(exp_avg, sizes)]
        exp_avg_sq = [_alias(t, "exp_avg_sq", (state_dtype,), dev, n) for t, n in zip(exp_avg_sq, sizes)]
        if eight != (exp_avg_scale is not None) or eight != (exp_avg_sq_scale is not None):
            raise ValueError("8-bit moments, and only they, come with exp_avg_scale and exp_avg_sq_scale")
        if eight:
            exp_avg_scale, exp_avg_sq_scale = list(exp_avg_scale), list(exp_avg_sq_scale)
            if len(exp_avg_scale) != len(params) or len(exp_avg_sq_scale) != len(params):
                raise ValueError("exp_avg_scale and exp_avg_sq_scale need one tensor per parameter")
            exp_avg_scale = [_alias(t, "exp_avg_scale", (torch.float32,), dev, n) for t, n in zip(exp_avg_scale, blocks)]
            exp_avg_sq_scale = [_alias(t, "exp_avg_sq_scale", (torch.float32,), dev, n)
                                for t, n in zip(exp_avg_sq_scale, blocks)]
    else:
        if exp_avg_scale is not None or exp_avg_sq_scale is not None:
            raise ValueError("scales are given together with the moments")
        zeros = lambda: [torch.zeros(p.shape, dtype=torch.uint8, device=dev).view(state_dtype) if eight  # noqa: E731
                         else torch.zeros(p.shape, dtype=torch.float32, device=dev) for p in params]
        exp_avg, exp_avg_sq = zeros(), zeros()
        if eight:
            exp_avg_scale, exp_avg_sq_scale = ([torch.zeros(b, device=dev) for b in blocks] for _ in range(2))
        made = [*exp_avg, *exp_avg_sq, *(exp_avg_scale or ()), *(exp_avg_sq_scale or ())]
    decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(params)
    if len(decay) != len(params):
        raise ValueError("weight_decay must be a number or one per parameter")
    buffers = [t for group in (params, copies, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale) if group is not None
               for t in group if t.numel()]
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in buffers)
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        raise ValueError("the tensors of a plan must not overlap")
    return AdamWPlan(params, copies, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, [float(d) for d in decay], made)


def _device_scalar(t, name, dtype, device):
    if t.dtype != dtype or t.numel() != 1 or t.device != device:
        raise TypeError(f"{name} must be a number or a one-element {dtype} tensor on the parameters' device")
    return t.data_ptr()


def adamw_step(plan: AdamWPlan, grads: Sequence[Optional[torch.Tensor]], *, step, lr, betas=(0.9, 0.999), eps=1e-8,
               grad_scale: Optional[torch.Tensor] = None, seed: int = 0) -> None:
    """One AdamW step of the plan's tensors, in place.

    grads: one per parameter and of its shape, of one dtype (float32, float16 or bfloat16), or None to leave that parameter and its
    moments as they are.  step: the number of this step, from 1 on; lr: the learning rate; either may be a
    one-element device tensor (int64, float32), which is read when the step runs, so that a captured step can be
    replayed with others.  grad_scale: a one-element float32 device tensor the gradients are multiplied by (a clipping
    factor), or None.  seed: of the random rounding of 8-bit moments (hashed with the step)."""
    grads = list(grads)
    if len(grads) != len(plan.params):
        raise ValueError(f"{len(plan.params)} gradients are wanted, got {len(grads)}")
    gdt = next((g.dtype for g in grads if g is not None), torch.float32)
    if gdt not in DTYPE:
        raise TypeError("gradients must be float32, float16 or bfloat16")
    dev = plan.device
    pointers = (ctypes.c_void_p * len(grads))()
    for i, (g, shape) in enumerate(zip(grads, plan._shapes)):
        if g is None:
            continue
        if g.dtype != gdt or g.shape != shape or g.device != dev:
            raise ValueError(f"gradient {i} must have dtype {gdt} and shape {tuple(shape)} on {dev}")
        if not g.is_contiguous():
            grads[i] = g = g.contiguous()   # kept until the launch is enqueued
        pointers[i] = g.data_ptr() or None
    beta1, beta2 = betas
    step_at = _device_scalar(step, "step", torch.int64, dev) if isinstance(step, torch.Tensor) else None
    lr_at = _device_scalar(lr, "lr", torch.float32, dev) if isinstance(lr, torch.Tensor) else None
    scale_at = None if grad_scale is None else _device_scalar(grad_scale, "grad_scale", torch.float32, dev)
    stream = _stream(dev)
    with _on(dev):
        if stream not in plan._streams and not torch.cuda.is_current_stream_capturing():
            plan._used_on_current_stream(stream)
        _check("rlpl_adamw_step", library().rlpl_adamw_step(
            plan._host.ctypes.data, plan._device.data_ptr(), pointers, DTYPE[gdt], 0.0 if lr_at else float(lr), lr_at,
            float(beta1), float(beta2), float(eps), 1 if step_at else int(step), step_at, scale_at,
            int(seed) & 0xFFFFFFFF, stream))
    written = plan.params + (plan.copies or [])
    if any(g is None for g in grads):
        written = [p for p, g in zip(written, grads + grads) if g is not None]
    increment_version(written)   # a graph that saved an old value says so in its backward pass


# ------------------------------------------------------------------------------------------------------- gradients' norm

NORM = {2.0: 0, math.inf: 1}


def _without_gaps(t: torch.Tensor) -> bool:
    """Whether t's elements fill one run of memory, each once, in any order of its dimensions."""
    if t.is_contiguous():
        return True
    at = 1
    for stride, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != at:
            return False
        at *= n
    return True


_dtype_of = torch.Tensor.dtype.__get__


def _grad_list(grads, in_place):
    """(tensors to keep until the call returns, pointers, sizes, dtypes, device) of the gradients that are there.  All of a
    list is looked at by calls that are themselves compiled: 300 tensors take 60 us instead of 150."""
    kept = [g for g in grads if g is not None]
    if not kept:
        raise ValueError("grads holds no tensor")
    try:
        devices, dtypes = set(map(torch.Tensor.get_device, kept)), set(map(_dtype_of, kept))
        plain = len(devices) == 1 and min(devices) >= 0 and dtypes <= DTYPE.keys() and all(map(torch.Tensor.is_contiguous, kept))
    except (TypeError, RuntimeError):                          # no tensor; a sparse one, which has no strides
        plain = False
    if not plain:
        _refuse_or_pack(kept, in_place)
        dtypes = set(map(_dtype_of, kept))
    n = len(kept)
    codes = array("i", [DTYPE[dtypes.pop()]]) * n if len(dtypes) == 1 else array("i", [DTYPE[t] for t in map(_dtype_of, kept)])
    return (kept, array("Q", map(torch.Tensor.data_ptr, kept)), array("q", map(torch.Tensor.numel, kept)), codes, kept[0].device)


def _refuse_or_pack(kept, in_place):
    """Raises for a gradient that cannot be taken, and replaces those that have gaps."""
    for i, g in enumerate(kept):
        if not isinstance(g, torch.Tensor) or not g.is_cuda or g.dtype not in DTYPE or g.layout != torch.strided:
            raise TypeError(f"gradient {i} must be a dense float32, float16 or bfloat16 CUDA (HIP) tensor")
        if g.device != kept[0].device:
            raise ValueError(f"gradient {i} must be on {kept[0].device}, as the first one")
        if not _without_gaps(g):
            if in_place:
                raise ValueError(f"gradient {i} must fill its memory without gaps to be scaled in place")
            kept[i] = g.contiguous()


def _at(a: array) -> int:
    return a.buffer_info()[0]


def _norm_of(listed, max_norm, norm_type, eps, grad_scale, workspace):
    kept, pointers, sizes, dtypes, dev = listed
    if norm_type not in NORM:
        raise ValueError("norm_type must be 2 or inf")
    scale_at = None if grad_scale is None else _device_scalar(grad_scale, "grad_scale", torch.float32, dev)
    lib = library()
    norm = torch.empty((), dtype=torch.float32, device=dev)
    scale = None if max_norm is None else torch.empty_like(norm)
    ws = _scratch(lib.rlpl_grad_norm_workspace_bytes(_at(sizes), len(kept)), workspace, dev, "rlpl_grad_norm_workspace_bytes")
    wp, wn = _ws_ptr(ws)
    with _on(dev):
        _check("rlpl_grad_norm", lib.rlpl_grad_norm(
            _at(pointers), _at(sizes), _at(dtypes), len(kept), NORM[norm_type], scale_at,
            0.0 if max_norm is None else float(max_norm), float(eps), norm.data_ptr(), _ptr(scale), wp, wn, _stream(dev)))
    return norm, scale


def grad_norm(grads: Sequence[Optional[torch.Tensor]], *, max_norm=None, norm_type=2.0, eps=1e-6,
              grad_scale: Optional[torch.Tensor] = None, workspace=None):
    """The norm over all gradients (a 0-d float32 tensor), or with ``max_norm`` (norm, scale): scale =
    min(1, max_norm / (norm + eps)), the factor that clips the gradients, which ``adamw_step`` takes as its grad_scale.

    grads: float32, float16 or bfloat16 tensors of one device, of any strides, in any mixture, or None (passed over).
    norm_type: 2 or math.inf.  grad_scale: a one-element float32 device tensor that the gradients are meant to be
    multiplied by (1 / a loss scale): the norm is of the products, and scale includes it.  Squares are summed in float64.
    A NaN makes both NaN, an infinite norm a scale of 0."""
    norm, scale = _norm_of(_grad_list(grads, False), max_norm, norm_type, eps, grad_scale, workspace)
    return norm if max_norm is None else (norm, scale)


def _scale_listed(listed, scale):
    kept, pointers, sizes, dtypes, dev = listed
    at = _device_scalar(scale, "scale", torch.float32, dev)
    with _on(dev):
        _check("rlpl_grad_scale", library().rlpl_grad_scale(_at(pointers), _at(sizes), _at(dtypes), len(kept), at, _stream(dev)))
    increment_version(kept)   # a graph that saved an old value says so in its backward pass


def scale_grads(grads: Sequence[Optional[torch.Tensor]], scale: torch.Tensor) -> None:
    """Multiplies the gradients by ``scale``, a one-element float32 device tensor, in place (each element rounded once).
    grads as for ``grad_norm``; each fills its memory without gaps (a transposed one may), and no two overlap.
    A scale of exactly 1 writes nothing."""
    _scale_listed(_grad_list(grads, True), scale)


def clip_grads(grads: Sequence[Optional[torch.Tensor]], max_norm, *, norm_type=2.0, eps=1e-6, workspace=None) -> torch.Tensor:
    """Scales the gradients in place by min(1, max_norm / (norm + eps)) and returns their norm before that, a 0-d float32
    tensor.  Nothing is written where the norm is within max_norm; a NaN among the gradients makes all of them NaN, an
    infinity makes it NaN and the others 0.  Where ``adamw_step`` follows, ``grad_norm``'s scale saves this second pass over
    the gradients."""
    if max_norm is None:
        raise ValueError("max_norm must be a number")
    listed = _grad_list(grads, True)
    norm, scale = _norm_of(listed, max_norm, norm_type, eps, None, workspace)
    _scale_listed(listed, scale)
    return norm
