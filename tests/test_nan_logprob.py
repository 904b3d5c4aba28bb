"""Selective log-probabilities where a tile of the vocabulary holds a NaN, or nothing that counts."""
import pytest
import torch

import rl_post_loss_amd as rl
from test_linear_cross_entropy import DEV, E, make, on_device

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,H,V", [(3, 8, 5), (40, 64, 257), (200, 512, 2051), (64, 40, 1024)])
def test_nan_weight_row_at_the_end_of_the_vocabulary(n, H, V, dtype):
    for last in (1, 2, 3):
        c = make(n, H, V, dtype)
        c["w"][V - last] = NAN
        c["y"] = c["y"] % (V - 3)
        logp, lse = rl.selective_logprob_fwd(*on_device(c))
        assert torch.isnan(logp).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("first,count", [(0, 256), (256, 256), (512, 1)])
def test_nan_blocks_of_the_vocabulary(first, count):
    c = make(40, 64, 1088)
    c["w"][first:first + count] = NAN
    c["y"] = c["y"] % 100 + 900
    logp, lse = rl.selective_logprob_fwd(*on_device(c))
    assert torch.isnan(logp).all() and torch.isnan(lse).all()


def test_nan_beside_entries_taken_out():
    c = make(50, 64, 1024, seed=2)
    c["y"] = c["y"] % 16
    c["b"][16:] = -INF
    c["b"][1000] = NAN
    logp, _ = rl.selective_logprob_fwd(*on_device(c))
    assert torch.isnan(logp).all()


@pytest.mark.parametrize("first,count", [(0, 256), (256, 512), (300, 700), (768, 232)])
def test_tiles_taken_out_by_their_bias(first, count):
    """A bias of -inf over whole tiles: what is left, against float64.  Logits are off by at most (H + 4) E S with S =
    |h|.|W|^T + |b|, the log-sum-exp by the largest of those, 304 E for the sums and exponentials and 4 E |lse|."""
    c = make(60, 64, 1000, seed=3)
    left = torch.ones(1000, dtype=torch.bool)
    left[first:first + count] = False
    c["b"][~left] = -INF
    kept = torch.nonzero(left)[:, 0]
    c["y"] = kept[c["y"] % len(kept)]
    logp, lse = rl.selective_logprob_fwd(*on_device(c))
    h, w, b = c["h"].double(), c["w"].double()[left], c["b"].double()[left]
    want = torch.logsumexp(h @ w.t() + b, 1)
    zy = (h * c["w"].double()[c["y"]]).sum(1) + c["b"].double()[c["y"]]
    ez = ((64 + 4) * E * (h.abs() @ w.abs().t() + b.abs())).amax(1)
    tol = 1.01 * (ez + 304 * E + 4 * E * want.abs())
    assert ((lse.cpu().double() - want).abs() <= tol).all()
    assert ((logp.cpu().double() - (zy - want)).abs() <= tol + ez + 4 * E * (zy.abs() + want.abs())).all()
    g = torch.ones(60, device=DEV)
    dh, dw, db = rl.selective_logprob_bwd(*on_device(c), lse, g)
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all() and not dw[~left.to(DEV)].any() and not db[~left.to(DEV)].any()
