"""Statistics of logit rows in float64, counted from each row's largest logit: a row far from zero keeps its fractions."""
import torch


def statistics(z, T):
    """x = z / T, its largest b, lse, log-probabilities l = x - lse, p = exp(l) and entropies of rows with a finite largest logit."""
    x = z.double() / T
    b = x.amax(-1)
    d = x - b[..., None]
    L = torch.logsumexp(d, -1)
    l = d - L[..., None]
    p = l.exp()
    H = -torch.where(p > 0, p * l, 0.0).sum(-1)
    return x, b, b + L, L, l, p, H
