"""Token log-probabilities do not depend on a constant added to a row's logits.

Tolerances (eps = 2^-24; x = z / T; b the row's largest x; L = lse - b; all in natural units).  A term's exponent is off by 3 eps of its
own size at most: c's rounding, and one of an fma from the base c b, or those of (z - b) c.  What the terms count from, the rounded c b,
is what the results count from as well, and sums move from one base to another by the difference of the two; so no
share of |b| is left.  With D the distance of a term from the largest, 2^d is off by eps (2 + 3 D) relative, and
sum p D = H - L <= H.  s adds up to V / 256 terms a lane one after the other, moves to a larger maximum (4 eps, and 3 eps of the
distance, which the share that moves pays for with 2^-distance: 3 eps at most) at most once in 32 elements, and joins lanes,
wavefronts and pieces: E_s = (V / 256 * 1.3 + 120 + 3 (H + L)) eps bounds s's relative error.  Then

    logp = ln 2 (e_y - log2 s)    E_s + 6 eps (|x_y - b| + L)
    H = ln 2 (log2 s - t / s)     E_s (2 + H + L) + 6 eps (L + H)
    lse = ln 2 (c b + log2 s)     E_s + 6 eps (|b| + L + |lse|), its own size
"""
import pytest
import torch

import rl_post_loss_amd as rl
from test_token_logprobs import DEV, E32, check
from token_reference import statistics

pytestmark = pytest.mark.gpu


def free_of_the_base(z, y, T, out, top_k):
    logp, lse, entropy, top, index = out
    V = z.shape[-1]
    x, b, want, L, l, p, H = statistics(z, T)
    es = (V / 256 * 1.3 + 120 + 3 * (H + L)) * E32
    xy = x.gather(-1, y[:, None])[:, 0]
    check("logp", logp, l.gather(-1, y[:, None])[:, 0], es + 6 * E32 * ((xy - b).abs() + L))
    check("entropy", entropy, H, es * (2 + H + L) + 6 * E32 * (L + H))
    check("lse", lse, want, es + 6 * E32 * (b.abs() + L + want.abs()))
    best, order = torch.sort(z, dim=-1, descending=True, stable=True)
    assert torch.equal(index.cpu(), order[:, :top_k])
    xt = best[:, :top_k].double() / T
    check("top_logp", top, l.gather(-1, order[:, :top_k]), es[:, None] + 6 * E32 * ((xt - b[:, None]).abs() + L[:, None]))


# on both sides of 2^20 / c, where exponents change from c z - c b to (z - b) c
OFFSETS = [30.0, 300.0, 3e3, -3e3, 1e4, 1e5, -1e5, 7e5, 726817.25, 8e5, -8e5, 3e6]


@pytest.mark.parametrize("T", [1.0, 0.5, 0.03125])            # powers of two: x is a float32 too
@pytest.mark.parametrize("rows,V", [(1, 1000), (1, 4096), (1, 4097), (1, 50021), (1, 128256), (80, 16000)])
def test_offsets(rows, V, T):
    g = torch.Generator().manual_seed(V)
    noise = 3.0 * torch.randn(V, generator=g)
    rise = torch.arange(V) * (12.0 / V)                        # its maximum rises again and again
    z = torch.stack([(base + offset).float() for offset in OFFSETS for base in (noise, rise, noise * T, rise * T)])
    y = torch.randint(0, V, (len(z),), generator=g)
    y[1::4] = V - 1
    d, t = z.repeat(rows, 1).to(DEV), y.repeat(rows).to(DEV)
    out = rl.token_logprobs_fwd(d, t, temperature=T, top_k=5)
    n = len(z)
    free_of_the_base(z, y, T, [o[:n] for o in out], 5)
    free_of_the_base(z, y, T, [o[-n:] for o in out], 5)


@pytest.mark.parametrize("V", [4097, 20000, 128256])
def test_maxima_that_pass_from_one_form_of_the_exponent_to_the_other(V):
    """Rows that rise, or fall, over the border, from far below it, and from the lowest values."""
    edge = 2.0 ** 20 / 1.4426950408889634
    i = torch.arange(V, dtype=torch.float64)
    rows = [edge - 8 + 16 * i / V, edge + 8 - 16 * i / V, -edge - 8 + 16 * i / V, -edge + 8 - 16 * i / V,
            torch.where(i < V // 2, -edge * 2, edge * 2 + i / V), torch.where(i % 300 == 299, edge + 5 + i / V, edge - 3),
            torch.where(i < V - 3, torch.tensor(torch.finfo(torch.float32).min, dtype=torch.float64), edge + i / V),
            torch.where(i < V // 3, -3e38, torch.where(i < V // 2, 5.0, 3e5 + i / V))]
    z = torch.stack(rows).float()
    y = torch.tensor([V - 1, 0, V - 1, 0, V - 2, 299, V - 1, V - 5])
    free_of_the_base(z, y, 1.0, rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), top_k=5), 5)
    d, t = z.repeat(150, 1).to(DEV), y.repeat(150).to(DEV)
    free_of_the_base(z, y, 1.0, [o[-len(z):] for o in rl.token_logprobs_fwd(d, t, top_k=5)], 5)
