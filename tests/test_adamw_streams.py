"""A plan that is dropped while its step still waits on another stream than the plan was made on."""
import pytest
import torch

import rl_post_loss_amd as rl
from test_adamw import DEV, F8, HYPER, same, tensors

pytestmark = pytest.mark.gpu
SIZES = [70000, 0, 300, 1 << 20]


@pytest.mark.parametrize("state", [torch.float32, F8])
def test_moments_outlive_a_dropped_plan(state):
    """Memory that the making stream takes right after the drop keeps what is written there, and the step is the one
    that a plan kept alive takes."""
    p = [t.to(DEV) for t in tensors(SIZES, 1, 0.1)]
    q = [t.clone() for t in p]
    grads = [t.to(DEV) for t in tensors(SIZES, 2, 0.01)]
    kept = rl.adamw_plan(q, state_dtype=state)
    rl.adamw_step(kept, grads, step=1, seed=4, **HYPER)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    plan = rl.adamw_plan(p, state_dtype=state)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)       # the step waits some 50 ms
        rl.adamw_step(plan, grads, step=1, seed=4, **HYPER)
    dt = torch.float32 if state == torch.float32 else torch.uint8
    del plan
    taken = [torch.full((n,), 3, dtype=d, device=DEV) for n in SIZES if n for d in (dt, dt, torch.float32)]
    taken += [torch.full(((n + 255) // 256,), 3.0, device=DEV) for n in SIZES for _ in range(2)]
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in taken)
    for a, b in zip(p, q):
        same("param", a, b)


def test_a_stream_is_recorded_once():
    plan = rl.adamw_plan([torch.zeros(300, device=DEV)])
    seen = []
    plan._used_on_current_stream = lambda s: (seen.append(s), type(plan)._used_on_current_stream(plan, s))
    side = torch.cuda.Stream()
    for _ in range(2):
        rl.adamw_step(plan, [torch.ones(300, device=DEV)], step=1, **HYPER)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            rl.adamw_step(plan, [torch.ones(300, device=DEV)], step=1, **HYPER)
        torch.cuda.synchronize()
    assert seen == [side.cuda_stream]
