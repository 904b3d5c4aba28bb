"""8-bit moments over many steps, against exact ones.

Between two steps an element's root is a grid value a of its block (in units of the block's largest root).  A step
moves it by delta relative to that unit, and rounds it up with probability f = |delta| / d, d the distance to the
neighbour: the expectation stays, and the square's rises by f (1 - f) d^2 <= |delta| d.  d is at most an eighth of the
value in e4m3's normal range, and |delta| = r (1 - beta2) / 2 |X - X_top| with X = g^2 / v of the element and of the
block's largest, means of 1, so E|X - X_top| <= 2: a step adds at most (1 - beta2) / 8 of the moment, and the
1 / (1 - beta2) steps that a moment remembers an eighth.  Below, never: the rise is a variance.  The averages over the
elements are allowed five of their standard errors, which the sample gives.
"""
import pytest
import torch

import rl_post_loss_amd as rl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("beta2,kind", [(0.999, "gauss"), (0.999, "sparse"), (0.99, "gauss"), (0.95, "gauss")])
def test_moments_of_many_steps(beta2, kind):
    n, steps = 1 << 16, 2500 if beta2 == 0.999 else 600
    g = torch.Generator(device=DEV).manual_seed(3)
    spread = 1e-3 * torch.randn(n, device=DEV, generator=g).exp()
    plan = rl.adamw_plan([torch.zeros(n, device=DEV)], state_dtype=torch.float8_e4m3fn, weight_decay=0.0)
    m, v = (torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(2))
    for t in range(1, steps + 1):
        grad = torch.randn(n, device=DEV, generator=g) * spread
        if kind == "sparse":
            grad *= torch.rand(n, device=DEV, generator=g) < 0.02
        rl.adamw_step(plan, [grad], step=t, lr=0.0, betas=(0.9, beta2), seed=7)
        m.mul_(0.9).add_(grad.double(), alpha=0.1)
        v.mul_(beta2).add_(grad.double().square(), alpha=1 - beta2)
    held_m, held_v = (x.double() for x in plan.moments(0))
    off = (held_m - m) / spread
    assert abs(off.mean()) <= 5 * off.std() / n ** 0.5
    code = plan.exp_avg_sq[0].view(torch.uint8)
    normal = code >= 8                        # e4m3's normal values
    assert normal.sum() > 0.9 * n
    ratio = (held_v / v)[normal]
    error = 5 * ratio.std() / len(ratio) ** 0.5
    print(f"second moment held at {ratio.mean():.4f} of the exact one")
    assert 1.0 - error <= ratio.mean() <= 1.125 + error
