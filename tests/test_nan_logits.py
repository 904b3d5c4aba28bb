"""A logit that is not a number reaches the loss, wherever it stands: beside columns past the vocabulary's end, beside
entries that a bias of -inf takes out, and in a tile that holds nothing else.

What is NaN by the formulas is NaN in the result (a row's log-sum-exp over a NaN is NaN), so no tolerances are needed;
the rows and entries without one are compared with float64 under the operators' own tolerances.
"""
import pytest
import torch

import rl_post_loss_amd as rl
from test_linear_cross_entropy import DEV, IGNORE, make, on_device

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

# (n, H, V): vocabularies that end inside a lane's columns, a tile and at a tile's end, over both tile shapes
SIZES = [(3, 8, 5), (40, 64, 257), (40, 64, 300), (200, 512, 2051), (64, 40, 1024), (1500, 64, 20003)]


def spoiled(n, H, V, rows, dtype="bf16", seed=0):
    """A case whose weight rows `rows` are NaN, with no target in them."""
    c = make(n, H, V, dtype, seed=seed)
    c["w"][rows] = NAN
    bad = torch.zeros(V, dtype=torch.bool)
    bad[rows] = True
    good = torch.nonzero(~bad)[:, 0]
    c["y"] = good[c["y"] % len(good)]
    return c


def all_nan(c, **kw):
    args = on_device(c)
    loss, dh, dw, db = rl.linear_cross_entropy(*args, **kw)
    assert torch.isnan(loss) and torch.isnan(rl.linear_cross_entropy_fwd(*args, **kw))
    assert torch.isnan(dh[args[3] != IGNORE]).all() and torch.isnan(dw).all() and torch.isnan(db).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,H,V", SIZES)
def test_nan_weight_row_at_the_end_of_the_vocabulary(n, H, V, dtype):
    for last in (1, 2, 3):
        all_nan(spoiled(n, H, V, [V - last], dtype))


@pytest.mark.parametrize("first,count", [(0, 64), (64, 64), (0, 256), (256, 256), (1024, 64)])
@pytest.mark.parametrize("n,H,V", [(40, 64, 1088), (1500, 64, 20032)])
def test_nan_blocks_of_the_vocabulary(n, H, V, first, count):
    all_nan(spoiled(n, H, V, list(range(first, first + count))))


@pytest.mark.parametrize("V", [300, 1024])
def test_nan_beside_entries_taken_out(V):
    """Everything but the targets' columns and one NaN is taken out by the bias."""
    c = make(50, 64, V, seed=2)
    c["y"] = c["y"] % 16
    c["b"][16:] = -INF
    c["b"][V - 40] = NAN
    all_nan(c)
    c["b"][V - 40] = 0.0
    c["w"][V - 40, 3] = NAN
    all_nan(c)


def test_a_nan_row_of_the_hidden_states_stays_in_its_row():
    c = make(300, 64, 777, seed=4, ignored=0.2)
    c["y"][7] = 5
    clean = rl.linear_cross_entropy(*on_device(c), reduction="sum")
    c["h"][7, 9] = NAN
    args = on_device(c)
    loss, dh, dw, db = rl.linear_cross_entropy(*args, reduction="sum")
    assert torch.isnan(loss) and torch.isnan(rl.linear_cross_entropy_fwd(*args, reduction="sum"))
    others = torch.arange(300, device=DEV) != 7
    assert torch.isnan(dh[7]).all() and torch.equal(dh[others], clean[1][others])
    assert torch.isnan(dw).all() and torch.isnan(db).all()
