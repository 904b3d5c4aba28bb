"""Operators that score tokens, over the same C ABI.

* ``token_logprobs_fwd`` / ``token_logprobs_bwd``: log-probabilities of given tokens over rows of logits, with each row's
  entropy and its most likely tokens, and the gradient with respect to the logits;
* ``fp8_linear``: the logits of an output projection in 8 bits, with a scale for each block of 128;
* ``fp8_quantize``: its operands from wider ones.

As in the package's other entry points, this module marshals arguments only: every step runs in the library's HIP
kernels on the current stream of the tensors' device, without synchronising.
"""
from __future__ import annotations

import torch

from . import DTYPE, MASK_DTYPE, _check, _ws_ptr, library
from .training import GROUP, _dense, _empty, _on, _plain, _ptr, _scratch, _stream

__all__ = ["token_logprobs_fwd", "token_logprobs_bwd", "fp8_quantize", "fp8_linear"]


# ------------------------------------------------------------------------------------- token log-probabilities

def _rows_of(z: torch.Tensor):
    """(z, rows, inner, group stride, row stride): rows r at group_stride (r // inner) + row_stride (r % inner).  z is
    copied only where its rows do not lie so."""
    V, lead = z.shape[-1], z.shape[:-1]
    rows = z.numel() // V
    if z.is_contiguous():
        return z, rows, rows, 0, V
    if z.stride(-1) == 1 or V == 1:
        # the leading dimensions, from the innermost outwards, those of one row left out, neighbours joined
        dims = []
        for n, stride in zip(reversed(lead), reversed(z.stride()[:-1])):
            if n == 1:
                continue
            if dims and stride == dims[-1][0] * dims[-1][1]:
                dims[-1] = (dims[-1][0], dims[-1][1] * n) if dims[-1][0] else (0, dims[-1][1] * n)
            else:
                dims.append((stride, n))
        if len(dims) == 0:
            return z, rows, 1, 0, 0
        if len(dims) == 1:
            return z, rows, rows, 0, dims[0][0]
        if len(dims) == 2:
            return z, rows, dims[0][1], dims[1][0], dims[0][0]
    return z.contiguous(), rows, rows, 0, V


def _token_operands(logits, targets, mask):
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dtype not in DTYPE or logits.dim() < 1:
        raise TypeError("logits must be a float32, float16 or bfloat16 CUDA (HIP) tensor")
    z = _plain(logits)
    lead, dev = z.shape[:-1], z.device
    if not isinstance(targets, torch.Tensor) or targets.dtype != torch.int64 or targets.shape != lead or targets.device != dev:
        raise ValueError(f"targets must be an int64 {tuple(lead)} tensor on the logits' device")
    m = None
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype not in MASK_DTYPE or mask.shape != lead or mask.device != dev:
            raise ValueError(f"mask must be a bool, int8 or uint8 tensor of shape {tuple(lead)} on the logits' device")
        m = mask.contiguous()
    if z.numel() == 0:
        _check("token_logprobs", 2)
    z, *where = _rows_of(z)
    return z, targets.contiguous(), m, where


def token_logprobs_fwd(logits, targets, mask=None, *, temperature=1.0, top_k=0, workspace=None):
    """Log-probabilities of ``targets`` under softmax(logits / temperature), with the rows' entropies and most likely
    tokens, in one pass over the logits: (logp, lse, entropy, top_logp, top_index), None for the last two with top_k = 0.

    logits (*, V) float32, float16 or bfloat16, read where they lie as long as a row's elements are side by side and the
    rows take two strides at most (``logits[:, :-1]`` is not copied); targets int64 of the leading shape; mask bool, int8
    or uint8 of it, or None: rows of a zero are not read, and give 0 (indices -1).  logp, lse and entropy are float32 of
    the leading shape; top_logp (float32) and top_index (int64) have top_k <= 64 more columns (V up to 2^22 then), in falling
    order, the lowest index first among equal logits.  A target outside [0, V) gives logp = NaN; logits of -inf have probability 0.
    A row with a NaN or +inf gives NaN and indices of -1, one of -inf alone an lse of -inf and NaN in the other floats."""
    z, y, m, (rows, inner, group, stride) = _token_operands(logits, targets, mask)
    V, lead, dev, lib = z.shape[-1], z.shape[:-1], z.device, library()
    top_k = int(top_k)
    ws = _scratch(lib.token_logprobs_workspace_bytes(rows, V, top_k), workspace, dev, "token_logprobs_workspace_bytes")
    wp, wn = _ws_ptr(ws)
    logp = torch.empty_like(y, dtype=torch.float32)
    lse, entropy = torch.empty_like(logp), torch.empty_like(logp)
    top_logp = _empty((*lead, top_k), torch.float32, dev) if top_k else None
    top_index = _empty((*lead, top_k), torch.int64, dev) if top_k else None
    with _on(dev):
        _check("token_logprobs_fwd", lib.token_logprobs_fwd(
            z.data_ptr(), y.data_ptr(), _ptr(m), rows, V, inner, group, stride, DTYPE[z.dtype], float(temperature), top_k,
            logp.data_ptr(), lse.data_ptr(), entropy.data_ptr(), _ptr(top_logp), _ptr(top_index), wp, wn, _stream(dev)))
    return logp, lse, entropy, top_logp, top_index


def token_logprobs_bwd(logits, targets, mask, lse, entropy, grad_logp=None, grad_entropy=None, *, temperature=1.0):
    """The gradient of sum(grad_logp * logp) + sum(grad_entropy * entropy) with respect to the logits: dense, of their
    shape and dtype.  logits, targets, mask and temperature as in the forward, lse and entropy (float32) what it gave;
    entropy may be None without a grad_entropy; the two gradients are float32 of the leading shape, or None (zeros).
    Probabilities are as exact as lse (2^-24 |lse|), and formed anew where |lse| is 8192 or more."""
    z, y, m, (rows, inner, group, stride) = _token_operands(logits, targets, mask)
    lead, dev = z.shape[:-1], z.device
    held = {"lse": lse, "entropy": entropy, "grad_logp": grad_logp, "grad_entropy": grad_entropy}
    if lse is None or (grad_entropy is not None and entropy is None):
        raise ValueError("lse, and with a grad_entropy the entropy, must be the forward's")
    for name, t in held.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.shape != lead or t.device != dev:
            raise ValueError(f"{name} must be a float32 {tuple(lead)} tensor on the logits' device")
        held[name] = _dense(t)
    grad = _empty(z.shape, z.dtype, dev)
    with _on(dev):
        _check("token_logprobs_bwd", library().token_logprobs_bwd(
            z.data_ptr(), y.data_ptr(), _ptr(m), *(_ptr(t) for t in held.values()), rows, z.shape[-1], inner, group, stride,
            DTYPE[z.dtype], float(temperature), grad.data_ptr(), _stream(dev)))
    return grad


# ------------------------------------------------------------------------------------------------------- 8-bit products

def fp8_quantize(x, *, block_rows=1):
    """x (*, C) in 8 bits with a float32 scale for each 128 columns of a row (block_rows 1, as ``fp8_linear`` takes its
    input) or for each 128 x 128 (block_rows 128, x (R, C), as it takes its weight): (q, scale), q of x's shape and dtype
    float8_e4m3fn, scale (*, ceil(C / 128)) or (ceil(R / 128), ceil(C / 128)).  x float32, float16 or bfloat16."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in DTYPE or x.dim() < 1:
        raise TypeError("x must be a float32, float16 or bfloat16 CUDA (HIP) tensor")
    if block_rows not in (1, GROUP):
        raise ValueError(f"block_rows must be 1 or {GROUP}")
    if block_rows != 1 and x.dim() != 2:
        raise ValueError("x must be a matrix to be cut into squares")
    if x.numel() == 0:
        _check("fp8_quantize", 2)
    x = _plain(x)
    if not (x.dim() == 2 and (x.stride(1) == 1 or x.shape[1] == 1)):
        x = x.contiguous()
    C = x.shape[-1]
    rows = x.numel() // C
    ld = x.stride(0) if x.dim() == 2 else C
    groups = (C + GROUP - 1) // GROUP
    q = _empty(x.shape, torch.float8_e4m3fn, x.device)
    scale = _empty((*x.shape[:-1], groups) if block_rows == 1 else ((rows + GROUP - 1) // GROUP, groups), torch.float32,
                   x.device)
    with _on(x.device):
        _check("rlpl_fp8_quantize", library().rlpl_fp8_quantize(x.data_ptr(), rows, C, ld, DTYPE[x.dtype], block_rows,
                                                               q.data_ptr(), scale.data_ptr(), _stream(x.device)))
    return q, scale


def _fp8_operand(q, scale, name, scale_shape):
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype != torch.float8_e4m3fn:
        raise TypeError(f"{name} must be a float8_e4m3fn CUDA (HIP) tensor")
    if not isinstance(scale, torch.Tensor) or scale.dtype != torch.float32 or tuple(scale.shape) != scale_shape \
            or scale.device != q.device:
        raise ValueError(f"{name}_scale must be a float32 {scale_shape} tensor on {name}'s device")
    q = q.contiguous()
    return q if q.data_ptr() % 16 == 0 else q.clone(), scale.contiguous()


def fp8_linear(x, x_scale, weight, weight_scale, bias=None, *, out_dtype=torch.bfloat16, workspace=None):
    """(x * x_scale) . (weight * weight_scale)^T + bias of 8-bit operands with a scale for each block of 128: the logits
    of an output projection.  x (*, H) and weight (V, H) float8_e4m3fn, H a multiple of 16; x_scale float32
    (*, ceil(H / 128)), weight_scale float32 (ceil(V / 128), ceil(H / 128)), as ``rms_norm_fp8`` and ``fp8_quantize`` give
    them; bias (V,) of out_dtype, or None.  The result is (*, V) of out_dtype: bfloat16, float16 or float32.

    Sums are float32; for 16-bit outputs each aligned eight of K's products first loses what lies below 2^-13 of the largest of
    them (1.5e-5 of ordinary results, more beside an outlier column); float32 outputs lose nothing.  x and weight are
    read where they lie if they are dense and 16-byte aligned; otherwise each call copies them, a slice of a projection
    as well: make such a weight dense once."""
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor) or x.dim() < 1 or weight.dim() != 2 \
            or x.shape[-1] != weight.shape[1] or x.device != weight.device:
        raise ValueError("x (*, H) and weight (V, H) must be tensors that agree in H and device")
    if out_dtype not in DTYPE:
        raise TypeError("out_dtype must be float32, float16 or bfloat16")
    V, H = weight.shape
    lead, dev = x.shape[:-1], x.device
    if x.numel() == 0 or weight.numel() == 0:
        _check("fp8_linear", 2)
    n, blocks = x.numel() // H, (H + GROUP - 1) // GROUP
    x, xs = _fp8_operand(x, x_scale, "x", (*lead, blocks))
    w, ws_ = _fp8_operand(weight, weight_scale, "weight", ((V + GROUP - 1) // GROUP, blocks))
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype != out_dtype or tuple(bias.shape) != (V,) or bias.device != dev:
            raise ValueError(f"bias must be a ({V},) tensor of out_dtype on the operands' device")
        bias = _dense(bias)
    lib = library()
    ws = _scratch(lib.fp8_linear_workspace_bytes(n, H, V), workspace, dev, "fp8_linear_workspace_bytes")
    wp, wn = _ws_ptr(ws)
    out = _empty((*lead, V), out_dtype, dev)
    with _on(dev):
        _check("fp8_linear", lib.fp8_linear(x.data_ptr(), xs.data_ptr(), w.data_ptr(), ws_.data_ptr(), _ptr(bias), n, H, V,
                                            DTYPE[out_dtype], out.data_ptr(), wp, wn, _stream(dev)))
    return out
