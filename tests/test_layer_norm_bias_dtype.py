"""A float32 bias without a weight beside 16-bit inputs: its gradient is the float32 sum, not a 16-bit one widened.

Tolerance: (n + 35) eps sum |dy|, of the float32 sum over the rows (tests/test_layer_norm.py), and no rounding after it.
"""
import pytest
import torch

import rl_post_loss_amd as rl
from test_layer_norm import DEV, DT, backward_case, make

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,H", [(1, 5), (70, 264), (333, 1111), (9, 20000)])
def test_float32_bias_without_a_weight(n, H, dtype):
    c = make(n, H, dtype, "fp32", "b")
    x, dy = c["x"].to(DEV), c["dy"].to(DEV)
    b = c["b"].to(DEV).requires_grad_()
    xg = x.clone().requires_grad_()
    rl.layer_norm_autograd(xg, None, b).backward(dy)
    _, mean, rstd = rl.layer_norm_fwd(x, None, b.detach())
    assert b.grad.dtype == torch.float32
    backward_case(c, mean, rstd, (xg.grad, None, b.grad))
    direct = rl.layer_norm_bwd(dy, x, None, mean, rstd, bias_dtype=torch.float32)
    assert torch.equal(direct[0], xg.grad) and direct[1] is None and torch.equal(direct[2], b.grad)
    narrow = rl.layer_norm_bwd(dy, x, None, mean, rstd)[2]          # as without the argument
    assert narrow.dtype == DT[dtype] and torch.equal(narrow, b.grad.to(DT[dtype]))
    alone = rl.layer_norm_bwd(dy, x, None, mean, rstd, need_x=False, bias_dtype=torch.float32)
    assert alone[0] is None and torch.equal(alone[2], b.grad)


@gpu
def test_compiled_and_refused():
    c = make(40, 136, "bf16", "fp32", "b")
    x, dy, b = c["x"].to(DEV), c["dy"].to(DEV), c["b"].to(DEV).requires_grad_()
    compiled = torch.compile(lambda x, b: rl.layer_norm_autograd(x, None, b), fullgraph=True, backend="aot_eager")
    compiled(x, b).backward(dy)
    _, mean, rstd = rl.layer_norm_fwd(x, None, b.detach())
    assert torch.equal(b.grad, rl.layer_norm_bwd(dy, x, None, mean, rstd, bias_dtype=torch.float32)[2])
    w = torch.ones(136, dtype=torch.bfloat16, device=DEV)
    assert rl.layer_norm_bwd(dy, x, w, mean, rstd, bias_dtype=torch.bfloat16)[2].dtype == torch.bfloat16
    for weight, dtype in ((None, torch.float16), (None, torch.float64), (w, torch.float32)):
        with pytest.raises(TypeError, match="bias_dtype"):
            rl.layer_norm_bwd(dy, x, weight, mean, rstd, bias_dtype=dtype)


def test_the_fake_has_the_bias_dtype():
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        x, stat = torch.empty(3, 16, dtype=torch.bfloat16), torch.empty(3)
        op = torch.ops.rlpl.layer_norm_backward
        assert op(x, x, None, stat, stat, True, False, True, torch.float32)[2].dtype == torch.float32
        assert op(x, x, None, stat, stat, True, False, True)[2].dtype == torch.bfloat16
