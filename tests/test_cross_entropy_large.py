"""The cross entropy where its rows by hidden values have more than 2^18 tiles, against float64.

Tolerances are those of tests/test_linear_cross_entropy.py, evaluated in parts of the rows.
"""
import pytest
import torch

import rl_post_loss_amd as rl
from test_linear_cross_entropy import DEV, E, U, check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 230 << 30:
        pytest.skip("needs 230 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def test_more_than_2_18_tiles_of_hidden_values():
    n, H, V = (1 << 18) + 300, 65536, 300
    assert ((n + 255) // 256) * (H // 256) > 1 << 18
    g = torch.Generator(device=DEV).manual_seed(1)
    h = torch.empty(n, H, dtype=torch.bfloat16, device=DEV)
    for part in h.split(8192):
        part.copy_(torch.randn(part.shape, device=DEV, generator=g))
    w = (torch.randn(V, H, device=DEV, generator=g) * 2 / 256).bfloat16()
    y = torch.randint(0, V, (n,), device=DEV, generator=g)
    loss, dh, dw, _ = rl.linear_cross_entropy(h, w, None, y)
    u, wd = U["bf16"], w.double()
    total, e_total = torch.zeros((), dtype=torch.float64, device=DEV), torch.zeros((), dtype=torch.float64, device=DEV)
    want, tol, sums = (torch.zeros(V, H, dtype=torch.float64, device=DEV) for _ in range(3))
    sampled = {0, 128, (1 << 18) - 4096 * 3 + 5, 1 << 18, (1 << 18) + 255, n - 1}
    for r0 in range(0, n, 4096):
        hd, t = h[r0:r0 + 4096].double(), y[r0:r0 + 4096]
        at = torch.arange(len(t), device=DEV)
        z = hd @ wd.t()
        ez = (H + 4) * E * (hd.abs() @ wd.abs().t())
        lse = torch.logsumexp(z, 1)
        p = torch.exp(z - lse[:, None])
        e_lse = (p * ez).sum(1) + (V / 64 + 300) * E + 4 * E * lse.abs()
        zy = z[at, t]
        total += (lse - zy).sum()
        e_total += (ez[at, t] + e_lse + 4 * E * (lse.abs() + zy.abs())).sum()
        hit = torch.zeros_like(p)
        hit[at, t] = 1.0
        dz = p - hit
        e_dz = p * (ez + e_lse[:, None] + 4 * E * ((z - lse[:, None]).abs() + 1)) + 2 * E * (p + hit)
        e_dz = e_dz + u * (dz.abs() + e_dz)
        want += dz.t() @ hd
        tol += e_dz.t() @ hd.abs()
        sums += dz.abs().t() @ hd.abs()
        for r in sampled:
            if r0 <= r < r0 + 4096:
                i = r - r0
                bound = e_dz[i] @ wd.abs() + (V + 24) * E * (dz[i].abs() @ wd.abs())
                check(f"grad_hidden row {r}", dh[r], ((dz[i] @ wd / n).cpu(), (bound / n).cpu()), u)
    check("loss", loss, ((total / n).cpu(), (e_total / n + 2 * E * (total / n).abs()).cpu()))
    check("grad_weight", dw, ((want / n).cpu(), ((tol + (n + 24) * E * sums) / n).cpu()), u)
    assert all(torch.isfinite(part).all() and part.any(dim=1).all() for part in dh.split(16384))
