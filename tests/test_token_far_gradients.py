"""Gradients of token log-probabilities where lse is so large that float32 does not hold its fraction.

Rows of the type's lowest value (a mask that leaves nothing) have the gradient of a uniform distribution, and rows far from zero
that of the row moved to zero.  Tolerances (eps = 2^-24, x = z / T, b the largest x, L = lse - b, D = b - x): the row's sums as in
the forward pass but for a maximum that may rise with every eight (four) elements: E_s = (V / 256 * 3 + 120 + 3 (H + L)) eps, or V / 64 of a row up to 2048; a term's
log-probability l by E_s + 6 eps (D + L), p by that and 3 eps more; dz as in the other gradients' test.
"""
import math

import pytest
import torch

import rl_post_loss_amd as rl
from test_token_logprobs import DEV, DT, E32, check, rounding
from token_reference import statistics

pytestmark = pytest.mark.gpu


def gradient_case(z, y, T, g, h, dz):
    V = z.shape[-1]
    x, b, _, L, l, p, H = statistics(z, T)
    es = (V / (64 if V <= 2048 else 256) * 3 + 120 + 3 * (H + L))[:, None] * E32
    hit = (torch.arange(V)[None] == y[:, None]).double()
    g, h, H = g.double()[:, None], h.double()[:, None], H[:, None]
    low = torch.where(p > 0, l, 0.0)
    want = (g * (hit - p) - h * p * (low + H)) / T
    e_l = torch.where(p > 0, es + 6 * E32 * ((x - b[:, None]).abs() + L[:, None]), 0.0)
    # H is the forward's, by E_s (2 + H + L) + 6 eps (L + H) of its own test
    e_h = es * (2 + H + L[:, None]) + 6 * E32 * (H + L[:, None])
    tol = (g.abs() * p + h.abs() * p * (low + H).abs()) * (e_l + 4 * E32) + h.abs() * p * (e_l + e_h) \
        + 6 * E32 * (g.abs() * (hit + p) + h.abs() * p * (low.abs() + H.abs()))
    check("grad_logits", dz, want, 1.01 * tol / T + rounding(want, dz.dtype))


SIZES = [(1, 7), (3, 1000), (3, 2048), (3, 2049), (2, 5003), (5, 20000), (300, 5000), (1, 128256)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,V", SIZES)
def test_rows_of_the_types_lowest_value(rows, V, dtype):
    z = torch.randn(rows, V, generator=torch.Generator().manual_seed(V)).to(DT[dtype])
    z[::2] = torch.finfo(DT[dtype]).min
    y = torch.arange(rows) % V
    g, h = torch.randn(rows, generator=torch.Generator().manual_seed(1)), torch.full((rows,), 0.3)
    for T in (1.0, 0.5, 4.0):
        out = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), temperature=T)
        dz = rl.token_logprobs_bwd(z.to(DEV), y.to(DEV), None, out[1], out[2], g.to(DEV), h.to(DEV), temperature=T)
        gradient_case(z[::2], y[::2], T, g[::2], h[::2], dz[::2])
        # their sum over the vocabulary is zero; each of the V elements is off by its rounding at most
        assert (dz[::2].double().sum(-1).abs() <= 2 * (torch.finfo(DT[dtype]).eps + (V + 200) * E32) * g[::2].abs().double().to(DEV) / T
                + V * 2.0 ** -25).all()


@pytest.mark.parametrize("offset", [1e4, -1e4, 1e5, 1e6, -3e6])
@pytest.mark.parametrize("rows,V", SIZES)
def test_rows_far_from_zero(rows, V, offset):
    gen = torch.Generator().manual_seed(V)
    noise = 3 * torch.randn(rows, V, generator=gen)
    noise[0] = torch.arange(V) * (10.0 / V)                    # the maximum rises again and again
    z = (noise + offset).float()
    z[:, V // 2] = -math.inf
    y = torch.where(torch.arange(rows) % V == V // 2, 0, torch.arange(rows) % V)
    g, h = torch.randn(rows, generator=gen), torch.randn(rows, generator=gen)
    out = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV))
    dz = rl.token_logprobs_bwd(z.to(DEV), y.to(DEV), None, out[1], out[2], g.to(DEV), h.to(DEV))
    gradient_case(z, y, 1.0, g, h, dz)


@pytest.mark.parametrize("V", [900, 9000])
def test_through_autograd_beside_ordinary_rows_and_in_a_replayed_graph(V):
    z = torch.randn(6, V, generator=torch.Generator().manual_seed(2))
    z[1] += 5e4
    z[4] = torch.finfo(torch.float32).min
    y = torch.arange(6)
    leaf = z.to(DEV).requires_grad_()
    logp, entropy = rl.token_logprobs_autograd(leaf, y.to(DEV))
    (logp + entropy).sum().backward()
    one = torch.ones(6)
    gradient_case(z, y, 1.0, one, one, leaf.grad)
    d, t, ones = z.to(DEV), y.to(DEV), one.to(DEV)
    out = rl.token_logprobs_fwd(d, t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dz = rl.token_logprobs_bwd(d, t, None, out[1], out[2], ones, ones)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dz, leaf.grad)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_row_so_long_that_its_pieces_are_longer(dtype):
    """More than 1024 pieces of 8 vectors for each lane."""
    V = (1 << 24) + 8195 * (1 if dtype == "fp32" else 3)
    z = torch.randn(2, V, generator=torch.Generator().manual_seed(5)).to(DT[dtype])
    z[0] = torch.finfo(DT[dtype]).min
    y, one = torch.tensor([5, V - 1]), torch.ones(2)
    d, t = z.to(DEV), y.to(DEV)
    out = rl.token_logprobs_fwd(d, t)
    dz = rl.token_logprobs_bwd(d, t, None, out[1], out[2], one.to(DEV), one.to(DEV))
    for i in range(2):
        gradient_case(z[i:i + 1], y[i:i + 1], 1.0, one[:1], one[:1], dz[i:i + 1])


def test_a_tiny_temperature_whose_lse_is_infinite():
    z = torch.tensor([[1.0, 5.0, 2.0, 5.0]])
    y = torch.tensor([1])
    out = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), temperature=1e-38)
    assert out[1].isinf().all()
    dz = rl.token_logprobs_bwd(z.to(DEV), y.to(DEV), None, out[1], None, torch.full((1,), 1e-38, device=DEV), temperature=1e-38)
    assert torch.allclose(dz.cpu(), torch.tensor([[0.0, 0.5, 0.0, -0.5]]), rtol=1e-5, atol=0)


def test_impossible_rows_stay_nan():
    z = torch.zeros(3, 5000)
    z[0], z[1, 9] = -math.inf, math.nan
    y = torch.zeros(3, dtype=torch.int64)
    out = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV))
    dz = rl.token_logprobs_bwd(z.to(DEV), y.to(DEV), None, out[1], out[2], torch.ones(3, device=DEV))
    assert dz[:2].isnan().all() and dz[2].isfinite().all()
