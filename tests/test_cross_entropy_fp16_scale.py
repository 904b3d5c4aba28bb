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


@gpu
def test_float32_hidden_gradients_of_no_rows_and_in_a_replayed_graph():
    args = on_device(make(40, 64, 300, "fp16", ignored=1.1))
    out = rl.linear_cross_entropy(*args, hidden_grad_dtype=torch.float32)
    assert out[0] == 0 and out[1].dtype == torch.float32 and not out[1].any()
    sets = [on_device(make(40, 64, 300, "fp16", ignored=0.3, seed=s)) for s in range(4)]
    static = [t.clone() for t in sets[0]]
    call = lambda a: rl.linear_cross_entropy(*a, hidden_grad_dtype=torch.float32)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(static)
    for c in sets[1:]:
        for t, new in zip(static, c):
            t.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call(c)))


@gpu
@pytest.mark.parametrize("wanted", [(0,), (1,), (2,), (0, 2), (1, 2)])
def test_fp16_gradients_of_some_inputs(wanted):
    args = on_device(make(90, 64, 500, "fp16", ignored=0.2))
    leaves = [t.clone().requires_grad_(i in wanted) for i, t in enumerate(args[:3])]
    (256.0 * rl.linear_cross_entropy_autograd(*leaves, args[3], reduction="sum")).backward()
    need = dict(need_hidden=0 in wanted, need_weight=1 in wanted, need_bias=2 in wanted)
    direct = rl.linear_cross_entropy(*args, reduction="sum", weight_grad_dtype=torch.float32,
                                     hidden_grad_dtype=torch.float32, **need)
    for i, (t, g) in enumerate(zip(leaves, direct[1:])):
        assert (t.grad is None) == (i not in wanted)
        assert g is None or torch.equal(t.grad, (g * 256.0).half())
