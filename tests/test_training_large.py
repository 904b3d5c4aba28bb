"""The operators of a training step on tensors whose offsets pass 31 and 32 bits, checked on parts of the result.

Tolerances are those of the operators' own tests; the parts are chosen so that they can be computed in float64: sampled
rows of a layer norm, sampled vocabulary entries of a cross entropy with few rows, the ends of an AdamW tensor.
"""
import numpy as np
import pytest
import torch

import adamw_reference as ref
import rl_post_loss_amd as rl
from test_adamw import DEV, F8, HYPER, f32_bits, same
from test_layer_norm import forward_case, backward_case
from test_linear_cross_entropy import E, U, check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def randn(*shape, scale=1.0):
    """bf16 normal numbers, a part at a time."""
    out = torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.numel(), device=DEV, generator=g) * scale)
    return out


@pytest.mark.parametrize("rows,cols", [(66000, 65536), (600000, 7177)])
def test_layer_norm_past_32_bits(rows, cols):
    assert rows * cols > 1 << 32
    x = randn(rows, cols)
    w = randn(cols) + 1
    y, mean, rstd = rl.layer_norm_fwd(x, w, w)
    at = torch.tensor([0, 1, 32767, 65535, rows - 2, rows - 1], device=DEV)
    forward_case(x[at].cpu(), w.cpu(), w.cpu(), 1e-5, (y[at], mean[at], rstd[at]))
    del y
    # a gradient of zero in all other rows leaves the sampled ones to make the weight's and bias's
    dy = torch.zeros_like(x)
    dy[at] = randn(len(at), cols)
    dx, dw, db = rl.layer_norm_bwd(dy, x, w, mean, rstd)
    c = {"x": x[at].cpu(), "w": w.cpu(), "dy": dy[at].cpu()}
    backward_case(c, mean[at], rstd[at], (dx[at], None, None))
    # the sums over the other rows add zeros exactly: as many steps as sampled rows
    h = (c["x"].double() - mean[at].cpu().double()[:, None]) * rstd[at].cpu().double()[:, None]
    d = c["dy"].double()
    e_h = E * (2 * h.abs() + ((c["x"].double() - mean[at].cpu().double()[:, None]).abs() * rstd[at].cpu().double()[:, None]))
    want = (d * h).sum(0)
    tol = (d.abs() * e_h).sum(0) + (len(at) + 35) * E * (d * h).abs().sum(0)
    check("grad_weight", dw, (want, tol), U["bf16"])
    check("grad_bias", db, (d.sum(0), (len(at) + 35) * E * d.abs().sum(0)), U["bf16"])
    dx[at] = 0
    assert not dx.any()


def test_cross_entropy_past_31_bits():
    n, H, V = 40, 4096, 600000
    assert V * H > 1 << 31
    h, w = randn(n, H), randn(V, H, scale=2 / 64)
    y = torch.randint(0, V, (n,), device=DEV)
    y[0], y[1] = 0, V - 1
    loss, dh, dw, _ = rl.linear_cross_entropy(h, w, None, y)
    z = torch.cat([h.double() @ part.double().t() for part in w.split(20000)], 1)
    lse = torch.logsumexp(z, 1)
    zy = z.gather(1, y[:, None])[:, 0]
    ez = (H + 4) * E * torch.cat([h.abs().double() @ part.abs().double().t() for part in w.split(20000)], 1)
    p = torch.exp(z - lse[:, None])
    e_lse = (p * ez).sum(1) + (V / 64 + 300) * E + 4 * E * lse.abs()
    e_rows = ez.gather(1, y[:, None])[:, 0] + e_lse + 4 * E * (lse.abs() + zy.abs())
    want = (lse - zy).mean()
    check("loss", loss, (want.cpu(), (e_rows.mean() + 2 * E * want.abs()).cpu()))
    at = torch.unique(torch.cat([y, torch.tensor([0, 1, V // 2, V - 300, V - 1], device=DEV)]))
    hit = torch.zeros_like(p)
    hit[torch.arange(n, device=DEV), y] = 1.0
    dz = (p - hit) / n
    u = U["bf16"]
    e_dz = (p * (ez + e_lse[:, None] + 4 * E * ((z - lse[:, None]).abs() + 1)) + 2 * E * (p + hit)) / n
    e_dz = e_dz + u * (dz.abs() + e_dz)
    hd = h.double()
    got = (dz[:, at].t() @ hd, e_dz[:, at].t() @ hd.abs() + (n + 24) * E * (dz[:, at].abs().t() @ hd.abs()))
    check("grad_weight", dw[at], tuple(t.cpu() for t in got), u)
    wide, bound = torch.zeros(n, H, dtype=torch.float64, device=DEV), torch.zeros(n, H, dtype=torch.float64, device=DEV)
    for v0 in range(0, V, 20000):
        part = w[v0:v0 + 20000].double()
        wide += dz[:, v0:v0 + 20000] @ part
        bound += (e_dz[:, v0:v0 + 20000] + (V + 24) * E * dz[:, v0:v0 + 20000].abs()) @ part.abs()
    check("grad_hidden", dh, (wide.cpu(), bound.cpu()), u)


@pytest.mark.parametrize("state", [torch.float32, F8])
def test_adamw_past_32_bits(state):
    n = (1 << 32) + 4321
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    copy = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    tail = 4321 + 256 * 3           # the last elements, from a block's first on, across 2^32
    ends = [(0, 512), (n - tail, 768), (1 << 32, n - (1 << 32))]
    for i, (start, k) in enumerate(ends):
        p[start:start + k] = torch.randn(k, device=DEV)
        g[start:start + k] = torch.randn(k, device=DEV) * 0.01
    before = [(p[a:a + k].cpu().numpy(), g[a:a + k].float().cpu().numpy()) for a, k in ends]
    plan = rl.adamw_plan([p], state_dtype=state, weight_decay=0.1, copies=[copy])
    rl.adamw_step(plan, [g], step=1, seed=5, **HYPER)
    k1 = ref.coefficients(HYPER["lr"], HYPER["betas"], HYPER["eps"], 1)
    for (a, k), (p0, g0) in zip(ends, before):
        zero = np.zeros(k, np.float32)
        want, m, r, v = ref.step(p0, g0, zero, zero, k1, 0.1)
        same("param", p[a:a + k], f32_bits(want))
        same("copy", copy[a:a + k], torch.from_numpy(want).bfloat16())
        if state == F8:
            words = ref.random_words(5, 1, 0, k, a)
            for x, q, scale, u, root in ((m, plan.exp_avg[0], plan.exp_avg_scale[0], words & np.uint64(0xFFFF), False),
                                         (r, plan.exp_avg_sq[0], plan.exp_avg_sq_scale[0], words >> np.uint64(16), True)):
                code, sc = ref.encode(x, u, root)
                same("code", q.view(torch.uint8)[a:a + k].view(F8), code)
                same("scale", scale[a // 256:(a + k + 255) // 256], f32_bits(sc))
        else:
            same("exp_avg", plan.exp_avg[0][a:a + k], f32_bits(m))
            same("exp_avg_sq", plan.exp_avg_sq[0][a:a + k], f32_bits(v))
    assert not plan.exp_avg[0].view(torch.uint8 if state == F8 else torch.int32)[1024:1 << 20].any()
