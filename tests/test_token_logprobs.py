"""Log-probabilities of given tokens over logit rows, entropies, most likely tokens, and the gradient, against float64.

Tolerances (eps = 2^-24; x = z / T; b the row's largest x; L = lse - b >= 0, at most log V):

* An exponent d = c z - c b (c = log2(e) / T rounded once) is one fma from a rounded c b; both roundings of b are shared
  by the row and fall out of every result but for their own size.  A term 2^d is off by eps (2 + |d|) relative (the
  instruction's 1 ulp, d's rounding), which weighted by 2^d / s is at most 2 + log2(e) (H + L).  s adds up to V / 256 terms a lane one after the
  other, counts anew (4 eps each) at most once in 32 elements where the maximum grows, and joins lanes, wavefronts and
  pieces: E_s = (V / 256 * 1.2 + 100 + 2 (H + L)) eps bounds s's relative error.
* lse = ln 2 (c b + log2 s): E_s + 4 eps (|b| + |x|max c's share: |b|) + 4 eps L + eps |lse|;
  logp = ln 2 (c z - c b - log2 s): E_s + 4 eps (|x_y - b| + L + |b|).
* H = ln 2 (log2 s - t / s): E_s (2 + H + L) from s and t's sums and 4 eps (L + H).
* Gradients (lse and H are inputs, exact): l = x - lse off by eps (2 |x| + |l|), p = e^l by that and 4 eps + 2 eps |l|;
  dz by (|g| p + |h| p |l + H|) rel(p) + |h| p e_l + 6 eps (|g| (hit + p) + |h| p (|l| + |H|)), over T, and the output's rounding.
"""
import ctypes
import math

import pytest
import torch

import rl_post_loss_amd as rl

E32 = 2.0 ** -24
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
gpu = pytest.mark.gpu


def rounding(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs() + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -149)


def check(name, got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    both = got.isfinite() & want.isfinite()
    same = torch.where(both, (got - want).abs() <= tol, (got == want) | (got.isnan() & want.isnan()))
    assert same.all(), f"{name}: {int((~same).sum())} of {same.numel()} off; got {got[~same][:3]}, want {want[~same][:3]}"


def make(rows, V, dtype, seed=0, scale=3.0, masked=0.0):
    g = torch.Generator().manual_seed(seed + 7 * rows + V)
    z = (scale * torch.randn(rows, V, generator=g)).to(DT[dtype])
    mask = torch.rand(rows, generator=g) >= masked
    return z, torch.randint(0, V, (rows,), generator=g), mask


def statistics(z, T):
    x = z.double() / T
    b = x.amax(-1)
    lse = torch.logsumexp(x, -1)
    l = x - lse[..., None]
    p = l.exp()
    H = -torch.where(p > 0, p * l, 0.0).sum(-1)
    return x, b, lse, l, p, H


def forward_case(z, y, T, out, top_k=0, mask=None):
    """z (rows, V), y (rows,) on the host; out: the kernel's."""
    logp, lse, entropy, top_logp, top_index = out
    V = z.shape[-1]
    x, b, want, l, p, H = statistics(z, T)
    L = want - b
    on = torch.ones_like(y, dtype=torch.bool) if mask is None else mask
    zero = lambda t: torch.where(on.reshape(on.shape + (1,) * (t.dim() - 1)), t, torch.zeros_like(t))  # noqa: E731
    es = (V / 256 * 1.2 + 100 + 2 * (H + L)) * E32
    inside = (y >= 0) & (y < V)
    xy = x.gather(-1, y.clamp(0, V - 1)[..., None])[..., 0]
    want_logp = torch.where(inside, xy - want, torch.nan)
    check("lse", lse, zero(want), es + (8 * b.abs() + 4 * L + want.abs()) * E32)
    check("logp", logp, zero(want_logp), es + 4 * E32 * ((xy - b).abs() + L + b.abs()))
    check("entropy", entropy, zero(H), es * (2 + H + L) + 4 * E32 * (L + H))
    if not top_k:
        assert top_logp is None and top_index is None
        return
    # -0 and 0 are equal; a stable sort leaves the lowest index first
    best, index = torch.sort(z.float() + 0.0, dim=-1, descending=True, stable=True)
    best, index = best[..., :top_k], index[..., :top_k]
    assert top_index.dtype == torch.int64
    want_index = torch.where(on[..., None], index, -1)
    assert torch.equal(top_index.cpu(), want_index), (top_index.cpu()[(top_index.cpu() != want_index).any(-1)][:2],
                                                      want_index[(top_index.cpu() != want_index).any(-1)][:2])
    xt = best.double() / T
    tol = es[..., None] + 4 * E32 * ((xt - b[..., None]).abs().nan_to_num(posinf=0.0) + L[..., None] + b[..., None].abs())
    check("top_logp", top_logp, zero(xt - want[..., None]), tol)


SHAPES = [(1, 1), (1, 2), (3, 7), (2, 8), (5, 9), (4, 255), (7, 2048), (3, 2049), (9, 4104), (2, 12345), (1, 128256), (8, 50021),
          (300, 1000), (2000, 513), (1100, 8191), (1, 1000003),
          (1030, 131072), (1025, 131200), (2, 1 << 22)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,V", SHAPES)
def test_forward_against_float64(rows, V, dtype):
    if rows * V > 1e8 and dtype != "bf16":
        pytest.skip("the largest sizes in one type")
    z, y, mask = make(rows, V, dtype, masked=0.3)
    k = min(V, (0, 1, 5, 20, 64)[(rows + V) % 5])
    T = (1.0, 0.7, 1.5)[V % 3]
    out = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), mask.to(DEV), temperature=T, top_k=k)
    forward_case(z, y, T, out, k, mask)
    out = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), temperature=T, top_k=min(V, 20))
    forward_case(z, y, T, out, min(V, 20))


def patterns(V):
    i = torch.arange(V)
    g = torch.Generator().manual_seed(V)
    few = torch.full((V,), -math.inf)
    few[torch.randperm(V, generator=g)[:3]] = torch.tensor([1.0, 3.0, 2.0])
    lane = torch.randn(V, generator=g)
    lane[(i % 2048) < 8] += 100.0                         # the largest all fall to one lane's vectors
    lane4 = torch.randn(V, generator=g)
    lane4[(i % 1024) < 4] += 100.0
    piece = torch.randn(V, generator=g)
    piece[V // 2: V // 2 + 60] += 50.0
    return {"constant": torch.full((V,), 1.5), "rising": i / 64.0, "falling": -i / 64.0, "few allowed": few, "lane": lane,
            "lane of 4": lane4, "one place": piece, "zeros of both signs": torch.where(i % 2 == 0, 0.0, -0.0),
            "ties": torch.randint(-3, 4, (V,), generator=g).float(), "huge": torch.randn(V, generator=g) * 3e4,
            "lowest": torch.where(i % 5 == 0, 2.0, -65504.0), "last": torch.where(i == V - 1, 9.0, -1.0),
            "no finite but one": torch.where(i == V // 3, 0.5, -math.inf)}


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [70, 4099, 40000, 70001])
@pytest.mark.parametrize("copies", [1, 1030])              # a row in pieces, and a workgroup a row
def test_patterns_of_logits(V, dtype, copies):
    if copies > 1 and V >= 40000:
        copies = 80                                        # 13 patterns each
    rows = patterns(V)
    z = torch.stack(list(rows.values())).to(DT[dtype])
    y = torch.arange(len(rows)) * 3 % V
    for k in (1, 20, 64):
        out = rl.token_logprobs_fwd(z.repeat(copies, 1).to(DEV), y.repeat(copies).to(DEV), top_k=k)
        forward_case(z, y, 1.0, [t[:len(rows)] for t in out], k)
        forward_case(z, y, 1.0, [t[-len(rows):] for t in out], k)


@gpu
@pytest.mark.parametrize("V", [64, 511, 512, 513, 2047, 2048, 2049, 4096, 4097])
def test_equal_logits_of_short_rows(V):
    """More elements reach the bound than there is room for; of equal ones the first are the alternatives."""
    z = torch.zeros(8, V, dtype=torch.bfloat16)
    z[1] = -1.5
    z[2, ::2] = -0.0                                           # equal to 0
    z[3] = -math.inf
    z[3, V // 2:V // 2 + 3] = 2.0
    z[4, :V - 40] = -math.inf
    z[5] = torch.arange(V) % 2
    z[6] = torch.finfo(torch.bfloat16).min
    z[6, -1] = 0.0
    z[7] = torch.arange(V).flip(0) // 50
    k = 64
    order = torch.sort(z.float(), dim=-1, descending=True, stable=True).indices[:, :k]
    for at in (0, 1):                                          # rows that start between two vectors likewise
        y = torch.zeros(8, dtype=torch.int64)
        buffer = torch.zeros(8, V + 5, dtype=torch.bfloat16, device=DEV)
        buffer[:, at:at + V] = z.to(DEV)
        index = rl.token_logprobs_fwd(buffer[:, at:at + V], y.to(DEV), top_k=k)[4]
        assert torch.equal(index.cpu(), order), [i for i in range(8) if not torch.equal(index[i].cpu(), order[i])]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [65, 130, 333, 500, 1000, 2048, 4001])
def test_many_alternatives_of_short_rows(V, dtype):
    """Few lanes with elements, many alternatives, and rows most of which is -inf."""
    z = make(12, V, dtype)[0]
    z[4:8, torch.rand(V, generator=torch.Generator().manual_seed(V)) < 0.6] = -math.inf
    z[8:10] = (z[8:10] * 4).round() / 4                        # many equal ones
    z[10] = torch.linspace(-1000, 0, V).exp().to(z.dtype)      # bisection finds no middle
    z[11, V // 2:] += 500
    y = torch.zeros(12, dtype=torch.int64)
    for k in (20, 33, 48, 64):
        order = torch.sort(z.float(), dim=-1, descending=True, stable=True).indices[:, :k]
        index = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), top_k=k)[4].cpu()
        assert torch.equal(index, order), [i for i in range(12) if not torch.equal(index[i], order[i])]


@gpu
@pytest.mark.parametrize("rows,V", [(1, 5000), (1200, 5000), (1, 70001), (3, 70001), (2, 3000)])
def test_nan_and_infinite_logits(rows, V):
    z, y, _ = make(rows, V, "fp32")
    for where, bad in ((V - 679, math.nan), (0, math.inf), (17, math.nan)):
        w = z.clone()
        w[0, where] = bad
        logp, lse, entropy, top, index = rl.token_logprobs_fwd(w.to(DEV), y.to(DEV), top_k=4)
        assert logp[0].isnan() and lse[0].isnan() and entropy[0].isnan() and top[0].isnan().all() and (index[0] == -1).all()
        if rows > 1:
            forward_case(z[1:], y[1:], 1.0, [t[1:] for t in (logp, lse, entropy, top, index)], 4)
    w = z.clone()
    w[0] = math.nan
    assert (rl.token_logprobs_fwd(w.to(DEV), y.to(DEV), top_k=4)[4][0] == -1).all()
    w[0] = -math.inf                                       # no token is possible
    logp, lse, entropy, top, index = rl.token_logprobs_fwd(w.to(DEV), y.to(DEV), top_k=4)
    assert lse[0] == -math.inf and logp[0].isnan() and entropy[0].isnan() and top[0].isnan().all()
    assert index[0].tolist() == [0, 1, 2, 3]
    w[0, 77], y[0] = 4.0, 77                               # one is
    logp, lse, entropy, top, index = rl.token_logprobs_fwd(w.to(DEV), y.to(DEV), top_k=4)
    assert logp[0] == 0 and abs(float(lse[0]) - 4) <= 8 * E32 and entropy[0] == 0 and index[0].tolist() == [77, 0, 1, 2]
    assert top[0, 0] == 0 and (top[0, 1:] == -math.inf).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,V", [(1, 5003), (1100, 5003), (2, 70003), (2, 1001)])
def test_masks_of_the_types_lowest_value(rows, V, dtype):
    """Rows that are all of it give a uniform distribution; beside other logits it has probability 0."""
    low = torch.finfo(DT[dtype]).min
    z, y, _ = make(rows, V, dtype, seed=6)
    z[0] = low
    for T in (1.0, 0.6, 3.0):
        logp, lse, H, top, index = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), temperature=T, top_k=5)
        uniform = math.log(V)
        assert abs(float(logp[0]) + uniform) <= 200 * E32 * uniform and abs(float(H[0]) - uniform) <= 200 * E32 * uniform
        assert index[0].tolist() == [0, 1, 2, 3, 4] and ((top[0] + uniform).abs() <= 200 * E32 * uniform).all()
        want = torch.tensor(low, dtype=torch.float64) / T + uniform
        assert abs(float(lse[0]) - want.float().item()) <= 4 * E32 * abs(want) or float(lse[0]) == want.float().item()
    w = z.clone()
    w[0] = z[-1] if rows > 1 else torch.randn(V).to(DT[dtype])
    w[0, ::3] = low
    y[0] = 1
    for T in (1.0, 0.6):
        out = rl.token_logprobs_fwd(w.to(DEV), y.to(DEV), temperature=T, top_k=20)
        forward_case(w[:1], y[:1], T, [t[:1] for t in out], 20)
        one = torch.ones(rows, device=DEV)
        dz = rl.token_logprobs_bwd(w.to(DEV), y.to(DEV), None, out[1], out[2], one, one, temperature=T)
        backward_case(w[:1], y[:1], T, out[1][:1].cpu(), out[2][:1].cpu(), one[:1].cpu(), one[:1].cpu(), dz[:1])
        assert (dz[0, ::3] == 0).all()


@gpu
@pytest.mark.parametrize("T", [1e-3, 1e-30, 1e-38, 1e3, 1e38])
def test_extreme_temperatures(T):
    z, y, _ = make(3, 4000, "fp32", seed=8)
    y[0] = z[0].argmax()
    out = rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), temperature=T, top_k=3)
    x = z.double() / torch.tensor(T, dtype=torch.float32).double()
    l = x - torch.logsumexp(x, -1, keepdim=True)
    want = l.gather(-1, y[:, None])[:, 0]
    L = (torch.logsumexp(x, -1) - x.amax(-1))
    tol = (4000 / 256 * 1.2 + 150 + 4 * L) * E32 + 8 * E32 * (want.abs() + (x.amax(-1).abs() if T > 1e-10 else 0.0))
    fits = want.abs() < 3e38
    assert ((out[0].cpu().double() - want).abs() <= tol)[fits].all() and out[0].cpu()[~fits].isinf().all()
    assert torch.equal(out[4].cpu(), torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :3])


@gpu
def test_masked_rows_are_not_read_and_targets_outside():
    z, y, _ = make(1500, 777, "bf16")
    mask = torch.arange(1500) % 3 > 0
    w = z.clone()
    w[~mask] = math.nan
    y[1], y[2], y[0] = -100, 777, 10 ** 12
    for kind in (torch.bool, torch.int8, torch.uint8):
        m = mask.to(kind)
        for n in (1500, 6):
            out = rl.token_logprobs_fwd(w[:n].to(DEV), y[:n].to(DEV), m[:n].to(DEV), top_k=3)
            forward_case(z[:n], y[:n], 1.0, out, 3, mask[:n])
            assert out[0][1].isnan() and out[0][2].isnan() and out[0][0] == 0
            g = torch.ones(n, device=DEV)
            dz = rl.token_logprobs_bwd(w[:n].to(DEV), y[:n].to(DEV), m[:n].to(DEV), out[1], out[2], g, g)
            assert (dz[~mask[:n].to(DEV)] == 0).all() and dz.isfinite().all()
    none = rl.token_logprobs_fwd(w.to(DEV), y.to(DEV), torch.zeros(1500, dtype=torch.bool, device=DEV), top_k=3)
    assert all((t == 0).all() for t in none[:4]) and (none[4] == -1).all()


@gpu
def test_rows_where_they_lie():
    base, _, _ = make(6 * 11, 1003, "bf16", seed=3)
    base = base.view(6, 11, 1003).to(DEV)
    y = torch.randint(0, 900, (6, 11), generator=torch.Generator().manual_seed(0)).to(DEV)
    views = {"shifted": (base[:, :-1], y[:, :-1]), "later": (base[:, 1:], y[:, 1:]), "cut vocabulary": (base[..., :900], y),
             "cut off 16 bytes": (base[..., 3:950], y), "every second": (base[::2, ::3], y[::2, ::3]),
             "turned": (base.transpose(0, 1), y.t()), "one sequence": (base[2], y[2]), "one row": (base[2, 5], y[2, 5]),
             "expanded": (base[:1].expand(6, 11, 1003), y), "expanded row": (base[:, :1].expand(6, 11, 1003), y),
             "vocabulary not last": (base.permute(2, 0, 1).contiguous().permute(1, 2, 0), y),
             "four dimensions": (base.view(3, 2, 11, 1003)[:, :, :-1], y.view(3, 2, 11)[:, :, :-1]),
             "three strides": (base.view(3, 2, 11, 1003)[:, :1, :-1].expand(3, 4, 10, 1003), y.view(3, 2, 11)[:, :1, :-1].expand(3, 4, 10))}
    for name, (z, t) in views.items():
        dense = z.contiguous()
        out = rl.token_logprobs_fwd(z, t, top_k=5)
        V = z.shape[-1]
        assert out[0].shape == t.shape and out[4].shape == (*t.shape, 5), name
        flat = [o.reshape(-1, *o.shape[t.dim():]) for o in out]
        forward_case(dense.reshape(-1, V).cpu(), t.reshape(-1).cpu(), 1.0, flat, 5)
        g = torch.randn(t.shape, device=DEV)
        a = rl.token_logprobs_bwd(z, t, None, out[1], out[2], g, g)
        b = rl.token_logprobs_bwd(dense, t.contiguous(), None, out[1], out[2], g, g)
        assert a.is_contiguous() and a.shape == z.shape and torch.equal(a, b), name


def backward_case(z, y, T, lse, H, g, h, dz):
    x = z.double() / T
    V = z.shape[-1]
    lse, H = lse.double()[:, None], H.double()[:, None]
    g = torch.zeros_like(lse) if g is None else g.double()[:, None]
    h = torch.zeros_like(lse) if h is None else h.double()[:, None]
    l = x - lse
    p = l.exp()
    hit = (torch.arange(V)[None] == y[:, None]).double()
    low = torch.where(p > 0, l, 0.0)
    want = (g * (hit - p) - h * p * (low + H)) / T
    e_l = torch.where(p > 0, E32 * (2 * x.abs() + l.abs()), 0.0)
    rel = e_l + (4 + 2 * low.abs()) * E32
    tol = (g.abs() * p + h.abs() * p * (low + H).abs()) * rel + h.abs() * p * e_l \
        + 6 * E32 * (g.abs() * (hit + p) + h.abs() * p * (low.abs() + H.abs()))
    check("grad_logits", dz, want, tol / T + rounding(want, dz.dtype))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,V", SHAPES)
def test_backward_against_float64(rows, V, dtype):
    if rows * V > 1e8:
        pytest.skip("sizes of the forward's pieces")
    z, y, _ = make(rows, V, dtype, seed=1)
    z[:, V // 3] = -math.inf if V > 2 else z[:, V // 3]
    if rows > 2:
        y[1] = -1                                          # no one-hot term
    T = (1.0, 0.7, 1.5)[V % 3]
    d, t = z.to(DEV), y.to(DEV)
    _, lse, H, _, _ = rl.token_logprobs_fwd(d, t, temperature=T)
    gen = torch.Generator().manual_seed(rows)
    g, h = torch.randn(rows, generator=gen), 0.3 * torch.randn(rows, generator=gen)
    for a, b in ((g, h), (g, None), (None, h), (None, None)):
        dz = rl.token_logprobs_bwd(d, t, None, lse, H if b is not None else None, None if a is None else a.to(DEV),
                                   None if b is None else b.to(DEV), temperature=T)
        assert dz.dtype == DT[dtype]
        backward_case(z, y, T, lse.cpu(), H.cpu(), a, b, dz)


@gpu
def test_autograd_against_torch_and_differences():
    z, y, mask = make(2 * 9, 67, "fp32", masked=0.3)
    z, y, mask = z.view(2, 9, 67), y.view(2, 9), mask.view(2, 9)
    gen = torch.Generator().manual_seed(4)
    g, h = torch.randn(2, 9, generator=gen).double(), torch.randn(2, 9, generator=gen).double()
    leaf = z.to(DEV).requires_grad_()
    logp, entropy = rl.token_logprobs_autograd(leaf, y.to(DEV), mask.to(DEV), temperature=0.8)
    ((logp * g.float().to(DEV)).sum() + (entropy * h.float().to(DEV)).sum()).backward()

    def f(a):
        l = torch.log_softmax(a / 0.8, -1)
        return (mask * (g * l.gather(-1, y[..., None])[..., 0] - h * (l.exp() * l).sum(-1))).sum()

    wide = z.double().requires_grad_()
    f(wide).backward()
    got = leaf.grad.cpu().double()
    # terms of at most |g| + |h| (|l| + H) <= 4 + 4 * 30, each off by a few eps times |x| <= 16
    assert ((got - wide.grad).abs() <= 1000 * E32 * 16).all()
    v, t = torch.randn(z.shape, generator=gen, dtype=torch.float64), 1e-5
    diff = (f(wide.detach() + t * v) - f(wide.detach() - t * v)) / (2 * t)
    assert abs((got * v).sum() - diff) <= 1e-5 * (1 + (got * v).abs().sum())
    assert (got[~mask] == 0).all()


@gpu
def test_autograd_single_outputs_slices_and_tracing():
    z, y, _ = make(3 * 6, 130, "bf16", seed=9)
    leaf = z.view(3, 6, 130).to(DEV).requires_grad_()
    t = y.view(3, 6).to(DEV)[:, 1:]
    logp, entropy = rl.token_logprobs_autograd(leaf[:, :-1], t)
    logp.sum().backward(retain_graph=True)
    a = leaf.grad.clone()
    assert (a[:, -1] == 0).all()
    out = rl.token_logprobs_fwd(leaf.detach()[:, :-1], t)
    one = torch.ones_like(logp)
    assert torch.equal(a[:, :-1], rl.token_logprobs_bwd(leaf.detach()[:, :-1], t, None, out[1], None, one))
    leaf.grad = None
    entropy.sum().backward()
    assert torch.equal(leaf.grad[:, :-1], rl.token_logprobs_bwd(leaf.detach()[:, :-1], t, None, out[1], out[2], None, one))
    traced = torch.compile(lambda q: rl.token_logprobs_autograd(q, t)[0], fullgraph=True, backend="aot_eager")
    assert torch.equal(traced(leaf.detach()[:, :-1]), out[0])
    with pytest.raises(RuntimeError):                      # a second derivative
        leaf.grad = None
        g, = torch.autograd.grad(rl.token_logprobs_autograd(leaf, y.view(3, 6).to(DEV))[0].sum(), leaf, create_graph=True)
        g.sum().backward()


@gpu
@pytest.mark.parametrize("V", [3001, 30011, 80021])      # a wavefront a row, a workgroup, pieces
def test_equal_bits_another_stream_and_a_replayed_graph(V):
    z, y, mask = make(5, V, "fp16", masked=0.2)
    d, t, m = z.to(DEV), y.to(DEV), mask.to(DEV)
    ref = rl.token_logprobs_fwd(d, t, m, top_k=7)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(rl.token_logprobs_fwd(d, t, m, top_k=7), ref))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = rl.token_logprobs_fwd(d, t, m, top_k=7)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    one = torch.ones(5, device=DEV)
    with torch.cuda.graph(graph):
        out = rl.token_logprobs_fwd(d, t, m, top_k=7)
        dz = rl.token_logprobs_bwd(d, t, m, out[1], out[2], one, one)
    for i in range(3):
        d.copy_(torch.randn(5, V, device=DEV) * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        ref = rl.token_logprobs_fwd(d, t, m, top_k=7)
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
        assert torch.equal(dz, rl.token_logprobs_bwd(d, t, m, ref[1], ref[2], one, one))


@gpu
def test_a_given_workspace():
    z, y, _ = make(3, 140000, "bf16")
    nbytes = rl.library().token_logprobs_workspace_bytes(3, 140000, 9)
    ws = torch.full((nbytes + 256,), 255, dtype=torch.uint8, device=DEV)
    forward_case(z, y, 1.0, rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), top_k=9, workspace=ws), 9)
    with pytest.raises(rl.RlplError):
        rl.token_logprobs_fwd(z.to(DEV), y.to(DEV), top_k=9, workspace=ws[:300])


@gpu
def test_past_32_bits_of_elements():
    rows, V = 17000, 131073
    z = torch.zeros(rows, V, dtype=torch.bfloat16, device=DEV)
    tail, y, _ = make(4, V, "bf16", seed=2)
    z[-4:] = tail.to(DEV)
    t = torch.zeros(rows, dtype=torch.int64, device=DEV)
    t[-4:] = y.to(DEV)
    out = rl.token_logprobs_fwd(z, t, top_k=3)
    forward_case(tail, y, 1.0, [o[-4:] for o in out], 3)
    forward_case(torch.zeros(1, V), torch.zeros(1, dtype=torch.int64), 1.0, [o[:1] for o in out], 3)
    g = torch.ones(rows, device=DEV)
    dz = rl.token_logprobs_bwd(z, t, None, out[1], out[2], g, g)
    backward_case(tail, y, 1.0, out[1][-4:].cpu(), out[2][-4:].cpu(), g[:4].cpu(), g[:4].cpu(), dz[-4:])


@gpu
def test_refusals_of_tensors():
    z, y = torch.zeros(4, 8, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    for bad, error in [((z.cpu(), y), TypeError), ((z.int(), y), TypeError), ((z, y.int()), ValueError), ((z, y[:2]), ValueError),
                       ((z, y.cpu()), ValueError), ((z, y, y), ValueError), ((z, y, torch.ones(3, dtype=torch.bool, device=DEV)), ValueError),
                       ((z[:0], y[:0]), rl.RlplError), ((z[:, :0], y), rl.RlplError)]:
        with pytest.raises(error):
            rl.token_logprobs_fwd(*bad)
    for k in (-1, 9, 65):
        with pytest.raises(rl.RlplError):
            rl.token_logprobs_fwd(z, y, top_k=k)
    for T in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(rl.RlplError):
            rl.token_logprobs_fwd(z, y, temperature=T)
    s = torch.zeros(4, device=DEV)
    for bad in [(None, s, s, s), (s[:2], s, s, s), (s.double(), s, s, s), (s, None, s, s), (s, s, s.half(), s)]:
        with pytest.raises(ValueError):
            rl.token_logprobs_bwd(z, y, None, *bad)


def test_refusals_of_the_c_entries():
    lib = rl.library()
    P, odd = ctypes.c_void_p(0x7F0000000000), ctypes.c_void_p(0x7F0000000001)

    def fwd(**k):
        d = dict(z=P, y=P, m=None, rows=4, V=100, inner=4, gs=0, rs=100, dt=2, T=1.0, top=0, logp=P, lse=P, H=P, tl=None, ti=None,
                 ws=P, wn=1 << 40, stream=None)
        assert set(k) <= set(d)
        return lib.token_logprobs_fwd(*(d | k).values())

    def bwd(**k):
        d = dict(z=P, y=P, m=None, lse=P, H=P, g=P, h=P, rows=4, V=100, inner=4, gs=0, rs=100, dt=2, T=1.0, out=P, stream=None)
        assert set(k) <= set(d)
        return lib.token_logprobs_bwd(*(d | k).values())

    for f in (fwd, bwd):
        assert f() == 7 or torch.cuda.is_available()
        assert f(z=None) == 1 and f(y=None) == 1 and f(lse=None) == 1
        for rows in (0, -3, 1 << 31):
            assert f(rows=rows) == 2
        for V in (0, -1, (1 << 31) - 65535, 1 << 40):
            assert f(V=V) == 2
        assert f(inner=0) == 2 and f(inner=5) == 2 and f(gs=-1) == 2 and f(rs=-1) == 2
        assert f(rows=4, inner=1, gs=1 << 62) == 2 and f(rs=1 << 61) == 2 and f(rows=1 << 30, inner=1 << 30, rs=1 << 40) == 2
        assert f(dt=3) == 4 and f(T=1e-40) == 5 and f(T=0.0) == 5 and f(T=math.nan) == 5 and f(T=math.inf) == 5 and f(T=-1.0) == 5
        assert f(z=odd) == 3 and f(y=ctypes.c_void_p(0x7F0000000004)) == 3 and f(lse=odd) == 3 and f(H=odd) == 3
    assert fwd(top=3) == 1 and fwd(top=3, tl=P) == 1 and fwd(top=65, tl=P, ti=P) == 2 and fwd(top=-1) == 2
    assert fwd(top=101, tl=P, ti=P) == 2 and fwd(ws=None) == 6 and fwd(wn=8) == 6 and fwd(ws=ctypes.c_void_p(0x7F0000000010)) == 3
    assert fwd(logp=None) == 1 and fwd(logp=odd) == 3
    assert fwd(top=1, tl=P, ti=P, V=(1 << 22) + 1) == 2 and fwd(V=(1 << 22) + 1, rs=1 << 23) != 2
    assert bwd(out=None) == 1 and bwd(out=odd) == 3 and bwd(H=None) == 1 and bwd(g=odd) == 3 and bwd(h=odd) == 3
    size = lib.token_logprobs_workspace_bytes
    assert size(0, 5, 0) == 0 and size(5, 0, 0) == 0 and size(5, 5, 6) == 0 and size(5, 1000, 65) == 0 and size(5, 1000, 64) > 0
    for rows in (1, 2, 7, 500, 1023, 1024, 5000):
        for V in (1, 100, 5000, 128256, 1 << 30):
            for k in (0, 1, 20, 64):
                if k <= V:
                    assert size(rows, V, k) % 256 == 0 and size(rows, V, k) <= 256 + rows * 64 * (16 + 8 * k) + 512
