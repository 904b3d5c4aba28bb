"""Gradients that are added to in place count as changed, as any tensor that is written in place does."""
import pytest
import torch

import rl_post_loss_amd as rl
from test_linear_cross_entropy import DEV, make, on_device

pytestmark = pytest.mark.gpu


def test_a_graph_that_saved_an_accumulated_gradient_says_so():
    args = on_device(make(30, 16, 50))
    dw, db = torch.ones(50, 16, device=DEV), torch.ones(50, device=DEV)
    p = torch.ones((), device=DEV, requires_grad=True)
    losses = [(p * dw).sum(), (p * db).sum()]
    rl.linear_cross_entropy(*args, grad_weight=dw, grad_bias=db)
    for loss in losses:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    versions = dw._version, db._version
    loss = (p * dw).sum()
    rl.linear_cross_entropy(*args, need_weight=False, grad_weight=dw, grad_bias=db)      # one of them is written
    assert (dw._version, db._version) == (versions[0], versions[1] + 1)
    loss.backward()
