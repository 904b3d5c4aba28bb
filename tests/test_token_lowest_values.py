"""Token log-probabilities of tokens that the lowest value of their type rules out: finite where z / T - lse is.

Tolerance (eps = 2^-24): such a log-probability is (z - b) / T by four float32 operations and two rounded constants, beside which the
row's sums vanish: 8 eps relative.  What is past float32 is -inf; close to it either is right.
"""
import math

import pytest
import torch

import rl_post_loss_amd as rl
from test_token_logprobs import DEV, DT, E32
from token_reference import statistics

pytestmark = pytest.mark.gpu
MOST = torch.finfo(torch.float32).max


def same(got, want):
    got = got.cpu().double()
    past = want < -MOST * (1 - 8 * E32)
    near = (got - want).abs() <= 8 * E32 * want.abs() + 1e-3
    assert torch.where(past, (got == -math.inf) | near, near).all(), (got[~near][:4], want[~near][:4])
    assert (got[want < -MOST * (1 + 8 * E32)] == -math.inf).all()


# a wavefront's rows, whole rows, rows in pieces
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,V", [(5, 70), (5, 4000), (5, 5000), (2, 70001), (300, 40000)])
def test_targets_and_alternatives_of_the_lowest_value(rows, V, dtype):
    low = torch.finfo(DT[dtype]).min
    for base in (0.0, -1e4, 0.7 * MOST if dtype != "fp16" else 6e4):   # the last: z - b is past the type
        z = torch.full((rows, V), low, dtype=DT[dtype])
        allowed = [0, V // 2, V - 1]
        z[:, allowed] = torch.tensor([base, base + 1, base - 1], dtype=torch.float32).to(DT[dtype])
        y = torch.full((rows,), 3)
        y[0] = V // 2
        for T in (1.0, 1.25, 4.0, 0.5):
            logp, lse, entropy, top, index = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), temperature=T, top_k=6)
            l = statistics(z, T)[4]
            assert not logp.isnan().any() and not entropy.isnan().any()
            same(logp, l.gather(-1, y[:, None])[:, 0])
            order = torch.sort(z.float(), dim=-1, descending=True, stable=True).indices[:, :6]
            assert torch.equal(index.cpu(), order)
            same(top, l.gather(-1, order))


def test_a_banned_token_times_its_mask_is_zero():
    z = torch.zeros(2, 5000)
    z[:, 7] = torch.finfo(torch.float32).min
    logp = rl.token_logprobs_fwd(z.to(DEV), torch.tensor([7, 8]).to(DEV))[0]
    assert (logp * torch.tensor([0.0, 1.0], device=DEV)).isfinite().all()


def test_impossible_tokens_and_rows_keep_their_values():
    """-inf has probability 0, a row with a NaN or +inf, or of -inf alone, none."""
    for V in (100, 5000, 70001):
        z = torch.zeros(5, V)
        z[0, 1] = -math.inf
        z[1, 9], z[2, 9] = math.nan, math.inf
        z[3] = -math.inf
        z[4] = torch.finfo(torch.float32).min
        z[4, 2] = math.inf
        logp = rl.token_logprobs_fwd(z.to(DEV), torch.ones(5, dtype=torch.int64, device=DEV))[0].cpu()
        assert logp[0] == -math.inf and logp[1:].isnan().all()
