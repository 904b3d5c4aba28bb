"""The cross entropy's gradients in float32, and the autograd form's fp16 gradients under a loss scale.

Scaled by a power of two and rounded once, an fp16 gradient is the float32 one's nearest fp16 value: equality, no
tolerance.  The float32 gradients have the operator's own tolerance without the output's rounding.
"""
import ctypes

import pytest
import torch

import rl_post_loss_amd as rl
from test_linear_cross_entropy import A, DEV, WS, check, expected, make, on_device

gpu = pytest.mark.gpu
SCALE = 65536.0


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,H,V,ignored", [(1, 8, 5, 0.0), (130, 64, 700, 0.3), (3000, 40, 900, 0.0), (17, 256, 9000, 0.2)])
def test_hidden_gradient_in_float32(n, H, V, ignored, dtype):
    c = make(n, H, V, dtype, ignored=ignored)
    if n == 1:
        c["y"][0] = 3
    args = on_device(c)
    want = expected(c, 1e-3)
    plain = rl.linear_cross_entropy(*args, z_loss=1e-3)
    for kw in ({}, dict(weight_grad_dtype=torch.float32), dict(need_weight=False)):
        out = rl.linear_cross_entropy(*args, z_loss=1e-3, hidden_grad_dtype=torch.float32, **kw)
        assert out[1].dtype == torch.float32 and torch.equal(out[0], plain[0])
        check("grad_hidden", out[1], want["grad_hidden"])
        if "need_weight" not in kw:            # the products' splits are the same: so are the sums
            assert torch.equal(out[1].to(args[0].dtype), plain[1])
    same = rl.linear_cross_entropy(*args, z_loss=1e-3, hidden_grad_dtype=args[0].dtype)
    assert all(torch.equal(a, b) for a, b in zip(same, plain))
    shaped = rl.linear_cross_entropy(args[0].view(1, n, H), *args[1:3], args[3].view(1, n), z_loss=1e-3,
                                     hidden_grad_dtype=torch.float32)
    assert shaped[1].shape == (1, n, H)


@gpu
def test_a_loss_scale_reaches_fp16_gradients_before_they_are_rounded():
    c = make(3000, 64, 5000, "fp16", ignored=0.1)
    args = on_device(c)
    leaves = [t.clone().requires_grad_() for t in args[:3]]
    (SCALE * rl.linear_cross_entropy_autograd(*leaves, args[3])).backward()
    direct = rl.linear_cross_entropy(*args, weight_grad_dtype=torch.float32, hidden_grad_dtype=torch.float32)
    small = 0
    for t, g in zip(leaves, direct[1:]):
        assert t.grad.dtype == torch.float16 and torch.equal(t.grad, (g * SCALE).half())
        small += int(((g.abs() < 2.0 ** -14) & (g != 0)).sum())
    assert small > 100000                      # below fp16's normal range without the scale
    leaves = [t.clone().requires_grad_() for t in args[:3]]
    rl.linear_cross_entropy_autograd(*leaves, args[3]).backward()
    for t, g in zip(leaves, rl.linear_cross_entropy(*args)[1:]):
        assert torch.equal(t.grad, g)          # without one: the direct call's
    compiled = torch.compile(lambda h: rl.linear_cross_entropy_autograd(h, *args[1:]), fullgraph=True, backend="aot_eager")
    h = args[0].clone().requires_grad_()
    (SCALE * compiled(h)).backward()
    alone = rl.linear_cross_entropy(*args, need_weight=False, need_bias=False, hidden_grad_dtype=torch.float32)
    assert torch.equal(h.grad, (alone[1] * SCALE).half())


def test_refusals_and_constants():
    assert rl.training.CE_HIDDEN_F32 == 1
    lib = rl.library()

    def call(flags, nbytes=64 << 20, dh=A + 0x500000):
        return rl.STATUS[lib.rlpl_linear_cross_entropy(
            flags, A, A + 0x100000, None, A + 0x300000, 64, 256, 1000, 1, -100, ctypes.c_float(0.0), 0, A + 0x400000, dh,
            A + 0x600000, None, 1, 0, WS, nbytes, None)]

    assert call(2) == call(1 << 31) == "RLPL_ERR_PARAM"
    assert call(1, nbytes=256) == "RLPL_ERR_WORKSPACE" and call(1, dh=A + 0x500008) == "RLPL_ERR_ALIGN"
    if not torch.cuda.is_available():
        assert call(0) == call(1) == "RLPL_ERR_DEVICE"


@gpu
def test_refusals_of_the_binding():
    args = on_device(make(8, 16, 40))
    for bad in (torch.float16, torch.float64):
        with pytest.raises(TypeError, match="hidden_grad_dtype"):
            rl.linear_cross_entropy(*args, hidden_grad_dtype=bad)
