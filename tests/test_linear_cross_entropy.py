"""The cross entropy of an output projection over a vocabulary, with its gradients, against float64.

Tolerances, per element, evaluated in float64 from the inputs (E = 2^-24, the most a float32 operation is off relative
to its result; u = half a step of the operand type, 2^-8 for bf16 and 2^-11 for fp16; `sub` the absolute rounding
below fp16's normals, 2^-25):

* logits: products of 16-bit operands are exact in float32; sums over H are off by at most (H + 4) E S, S = |h|.|W|^T + |b|.
* lse: the p-weighted logit error, (V / 256 + 300) E for the float32 sums over tiles and the exponentials, 4 E |lse|.
* a row's loss: both errors, 4 E (|lse| + |z_y|) and, of the penalty c lse^2, 2 c |lse| err(lse) + 4 E c lse^2.
  The loss sums rows in float64 and is rounded once.
* dz, at its scale: p's error relative: logit error + lse error + 4 E (|z - lse| + 1); the factor 1 + 2 c lse by
  2 c err(lse) + 4 E of itself; the rounding to the operand type, u |dz| + sub (at 256 times the value in fp16).
* grad_hidden: sum_v err(dz) |W|, (V + 24) E sum_v |dz||W| for the sums over K, pieces and splits, u |result| + sub.
* grad_weight and grad_bias: likewise over the N rows, (N + 24) E; rounded by u |result| + sub where they are 16 bits.
"""
import ctypes

import pytest
import torch

import rl_post_loss_amd as rl

DEV = "cuda:0"
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25}
IGNORE = -100
gpu = pytest.mark.gpu


def make(n, H, V, dtype="bf16", bias=True, ignored=0.0, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed * 7919 + n * 31 + H * 17 + V)
    y = torch.randint(0, V, (n,), generator=g)
    y[torch.rand(n, generator=g) < ignored] = IGNORE
    return {"h": torch.randn(n, H, generator=g).to(DT[dtype]),
            "w": (torch.randn(V, H, generator=g) * spread / H ** 0.5).to(DT[dtype]),
            "b": (0.5 * torch.randn(V, generator=g)).to(DT[dtype]) if bias else None, "y": y}


def on_device(c):
    return [None if c[k] is None else c[k].to(DEV) for k in "hwby"]


def expected(c, z_loss=0.0, reduction="mean", ignore=IGNORE):
    """Values and allowances: {name: (value, tolerance before the output's own rounding)}."""
    dtype = "bf16" if c["h"].dtype == torch.bfloat16 else "fp16"
    u, sub = U[dtype], SUB[dtype] / (256.0 if dtype == "fp16" else 1.0)
    keep = c["y"] != ignore
    h, w, y = c["h"].double()[keep], c["w"].double(), c["y"][keep]
    n, (V, H) = h.shape[0], w.shape
    b = torch.zeros(V, dtype=torch.float64) if c["b"] is None else c["b"].double()
    s = 1.0 / max(n, 1) if reduction == "mean" else 1.0
    z = h @ w.t() + b
    size = h.abs() @ w.abs().t() + b.abs().nan_to_num(posinf=0.0)
    ez = (H + 4) * E * size
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    e_lse = (p * ez).sum(1) + (V / 256 + 300) * E + 4 * E * lse.abs()
    at = torch.arange(n)
    zy = z[at, y]
    rows = lse - zy + z_loss * lse ** 2
    e_rows = ez[at, y] + e_lse + 4 * E * (lse.abs() + zy.abs()) + 2 * z_loss * lse.abs() * e_lse + 4 * E * z_loss * lse ** 2
    hit = torch.zeros_like(z)
    hit[at, y] = 1.0
    f = (1.0 + 2.0 * z_loss * lse)[:, None]
    e_f = (2.0 * z_loss * e_lse)[:, None] + 4 * E * f.abs()
    dz = f * p - hit
    far = (z - lse[:, None]).abs().nan_to_num(posinf=0.0)
    e_dz = f.abs() * p * (ez + e_lse[:, None] + 4 * E * (far + 1)) + e_f * p + 2 * E * (f.abs() * p + hit)
    e_dz = e_dz + u * (dz.abs() + e_dz) + sub
    loss = rows.sum() * s
    out = {"loss": (loss, e_rows.sum() * s + 2 * E * loss.abs())}
    dh = torch.zeros(c["h"].shape, dtype=torch.float64)
    e_dh = torch.zeros_like(dh)
    dh[keep] = s * (dz @ w)
    e_dh[keep] = s * (e_dz @ w.abs() + (V + 24) * E * (dz.abs() @ w.abs()))
    out["grad_hidden"] = (dh, e_dh)
    out["grad_weight"] = (s * (dz.t() @ h), s * (e_dz.t() @ h.abs() + (n + 24) * E * (dz.abs().t() @ h.abs())))
    out["grad_bias"] = (s * dz.sum(0), s * (e_dz.sum(0) + (n + 24) * E * dz.abs().sum(0)))
    return out


def check(name, got, want, u=0.0, sub=0.0):
    value, tol = want
    got = got.detach().cpu().double()
    assert got.shape == value.shape, name
    tol = 1.01 * tol + u * value.abs() + sub + 1e-45
    off = (got - value).abs()
    assert (off <= tol).all(), f"{name}: {int((~(off <= tol)).sum())} of {off.numel()} off, worst by " \
                               f"{(off / tol).nan_to_num(nan=float('inf')).max():.2f} of what is allowed"


def run_case(c, z_loss=0.0, reduction="mean", **kw):
    dtype = "bf16" if c["h"].dtype == torch.bfloat16 else "fp16"
    u, sub = U[dtype], SUB[dtype]
    args = on_device(c)
    out = rl.linear_cross_entropy(*args, z_loss=z_loss, reduction=reduction, **kw)
    alone = rl.linear_cross_entropy_fwd(*args, z_loss=z_loss, reduction=reduction)
    want = expected(c, z_loss, reduction)
    assert torch.equal(out[0], alone) or (torch.isnan(out[0]) and torch.isnan(alone))
    check("loss", out[0], want["loss"])
    check("grad_hidden", out[1], want["grad_hidden"], u, sub)
    f32 = out[2].dtype == torch.float32
    check("grad_weight", out[2], want["grad_weight"], 0 if f32 else u, 0 if f32 else sub)
    if c["b"] is None:
        assert out[3] is None
    else:
        check("grad_bias", out[3], want["grad_bias"], 0 if f32 else u, 0 if f32 else sub)
    assert not out[1][args[3] == IGNORE].any()
    return args, out


SHAPES = [(1, 8, 1), (1, 64, 300), (3, 8, 5), (2, 16, 255), (17, 40, 256), (64, 256, 1000), (129, 136, 257),
          (255, 72, 513), (256, 64, 512), (257, 128, 1025), (200, 512, 2051), (37, 64, 8200), (1030, 64, 300),
          (5, 2048, 777), (600, 24, 20000)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,H,V", SHAPES)
def test_against_float64(n, H, V, dtype):
    run_case(make(n, H, V, dtype))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ignored", [0.25, 0.75, 0.99])
def test_ignored_rows(ignored, dtype):
    c = make(700, 128, 1500, dtype, ignored=ignored, seed=3)
    args, out = run_case(c, z_loss=1e-2, reduction="sum")
    junk = args[0].clone()
    junk[args[3] == IGNORE] = float("nan")       # nothing of an ignored row is used
    again = rl.linear_cross_entropy(junk, *args[1:], z_loss=1e-2, reduction="sum")
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    kept = c["y"] != IGNORE                      # and the others give what they give alone
    run_case(dict(c, h=c["h"][kept], y=c["y"][kept]), z_loss=1e-2, reduction="sum")


@gpu
@pytest.mark.parametrize("z_loss", [0.0, 1e-4, 0.1])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_penalty_and_reduction_without_bias(z_loss, reduction):
    run_case(make(300, 64, 700, "bf16", bias=False, ignored=0.1), z_loss, reduction)
    run_case(make(300, 64, 700, "fp16", bias=False, ignored=0.1), z_loss, reduction, weight_grad_dtype=torch.float32)


@gpu
def test_no_row_counts():
    c = make(40, 32, 100, ignored=1.1)
    args, out = run_case(c)
    assert out[0] == 0 and not out[1].any() and not out[2].any() and not out[3].any()


@gpu
def test_another_ignore_index_and_targets_outside():
    c = make(50, 64, 400, ignored=0.3)
    args = on_device(c)
    other = args[3].clone()
    other[other == IGNORE] = 7
    c7 = dict(c, y=other.cpu())
    want = expected(c7, ignore=7)
    out = rl.linear_cross_entropy(args[0], args[1], args[2], other, ignore_index=7)
    check("loss", out[0], want["loss"])
    for bad in (400, -1, 1 << 40, -(1 << 40)):
        y = c["y"].clone()
        y[0] = bad
        loss, dh, dw, db = rl.linear_cross_entropy(*args[:3], y.to(DEV))
        assert torch.isnan(loss) and torch.isfinite(dw).all()
        assert torch.isnan(rl.linear_cross_entropy_fwd(*args[:3], y.to(DEV)))


@gpu
@pytest.mark.parametrize("V", [600, 1024])
def test_entries_taken_out_by_their_bias(V):
    """A bias of -inf, or of the type's lowest value, over whole tiles of the vocabulary and parts of others."""
    c = make(70, 64, V, seed=5)
    c["y"] = c["y"] % 40 + 530                       # targets that stay in
    for low in (float("-inf"), torch.finfo(torch.bfloat16).min):
        c["b"][:520] = low
        args, out = run_case(c)
        assert torch.isfinite(out[0]) and not out[2][:520].any() and not out[3][:520].any()
    c["y"][3] = 0
    c["b"][:520] = float("-inf")
    assert torch.isinf(rl.linear_cross_entropy_fwd(*on_device(c)))


@gpu
def test_large_logits():
    run_case(make(130, 256, 900, "bf16", spread=40.0))
    run_case(make(130, 256, 900, "fp16", spread=40.0))


@gpu
def test_accumulates_in_float32():
    a, b = make(300, 64, 500, seed=1, ignored=0.2), make(90, 64, 500, seed=2)
    b["w"], b["b"] = a["w"], a["b"]
    one = [rl.linear_cross_entropy(*on_device(c), weight_grad_dtype=torch.float32) for c in (a, b)]
    dw, db = torch.zeros(500, 64, device=DEV), torch.zeros(500, device=DEV)
    for c in (a, b):
        got = rl.linear_cross_entropy(*on_device(c), grad_weight=dw, grad_bias=db)
        assert got[2] is dw and got[3] is db
    assert torch.equal(dw, one[0][2] + one[1][2]) and torch.equal(db, one[0][3] + one[1][3])
    run_case(a, weight_grad_dtype=torch.float32)


@gpu
def test_more_than_one_piece_of_the_vocabulary():
    """17,000 rows: a piece is the 8192 columns it is at least, so 20,100 take three."""
    c = make(17000, 16, 20100, "bf16", ignored=0.97, seed=9)
    run_case(c)
    kept = c["y"] != IGNORE
    run_case(dict(c, h=c["h"][kept], y=c["y"][kept]))    # the same rows in a single piece


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ignored", [0.0, 0.4, 0.98])
def test_pieces_with_kept_and_formed_logits(ignored, dtype):
    """9,000 rows: pieces are 14,336 columns.  The logits that are kept are those of the first piece, of the second's
    first columns too, or all, by the rows that count.  Columns of equal weights and no target get equal gradients
    whichever way, and rows their own hidden gradient."""
    V = 36000
    c = make(9000, 32, V, dtype, ignored=ignored, seed=11)
    c["y"][c["y"] != IGNORE] = c["y"][c["y"] != IGNORE] % 500 + 17900      # in columns that have no equal without targets
    c["w"][18000:] = c["w"][:18000]
    c["b"][18000:] = c["b"][:18000]
    _, dh, dw, db = rl.linear_cross_entropy(*on_device(c), reduction="sum")
    free = torch.ones(18000, dtype=torch.bool, device=DEV)
    free[17900:] = free[:400] = False
    assert torch.equal(dw[:18000][free], dw[18000:][free]) and torch.equal(db[:18000][free], db[18000:][free])
    assert dw[17900:18400].any()
    rows = torch.cat([torch.arange(3), torch.arange(4000, 4040), torch.arange(8990, 9000)])
    want = expected(dict(c, h=c["h"][rows], y=c["y"][rows]), reduction="sum")["grad_hidden"]
    check("grad_hidden", dh[rows.to(DEV)], want, U[dtype], SUB[dtype])


@gpu
def test_wanted_gradients_leading_dimensions_and_repeats():
    c = make(120, 64, 333, ignored=0.2)
    args = on_device(c)
    full = rl.linear_cross_entropy(*args)
    shaped = rl.linear_cross_entropy(args[0].view(4, 30, 64), args[1], args[2], args[3].view(4, 30))
    assert shaped[1].shape == (4, 30, 64) and torch.equal(shaped[1].view(120, 64), full[1])
    strided = torch.empty(120, 100, dtype=torch.bfloat16, device=DEV)[:, 3:67]
    strided.copy_(args[0])
    assert all(torch.equal(a, b) for a, b in zip(rl.linear_cross_entropy(strided, *args[1:]), full))
    for flags in range(8):
        need = dict(need_hidden=bool(flags & 1), need_weight=bool(flags & 2), need_bias=bool(flags & 4))
        got = rl.linear_cross_entropy(*args, **need)
        assert torch.equal(got[0], full[0])
        for g, f, wanted in zip(got[1:], full[1:], need.values()):
            assert (g is not None) == wanted and (g is None or torch.equal(g, f))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(rl.linear_cross_entropy(*args), full))
    dirty = torch.full((rl.library().linear_cross_entropy_workspace_bytes(120, 64, 333, 1) + 256,), 255, dtype=torch.uint8,
                       device=DEV)                   # a workspace of any contents
    assert all(torch.equal(a, b) for a, b in zip(rl.linear_cross_entropy(*args, workspace=dirty), full))


@gpu
@pytest.mark.parametrize("n,H,V", [(1, 64, 9000), (40, 256, 9000), (700, 72, 30000), (1500, 264, 3000), (12000, 32, 25000)])
def test_the_hidden_gradient_alone(n, H, V):
    """Without the weight's gradient the product is split over the vocabulary in its own way."""
    c = make(n, H, V, ignored=0.98 if n > 2000 else 0.3, seed=6)
    if n == 1:
        c["y"][0] = V - 1
    _, dh, dw, db = rl.linear_cross_entropy(*on_device(c), need_weight=False, need_bias=False)
    assert dw is None and db is None
    check("grad_hidden", dh, expected(c)["grad_hidden"], U["bf16"])


@gpu
def test_a_bias_gradient_passed_without_a_bias_is_added_to():
    c = make(70, 40, 300, bias=False, seed=2)
    args = on_device(c)
    zero = torch.zeros(300, dtype=torch.bfloat16, device=DEV)
    want = rl.linear_cross_entropy(args[0], args[1], zero, args[3], weight_grad_dtype=torch.float32)
    dw, db = torch.ones(300, 40, device=DEV), torch.ones(300, device=DEV)
    out = rl.linear_cross_entropy(*args, grad_weight=dw, grad_bias=db)
    assert out[3] is db and torch.equal(db, 1.0 + want[3]) and torch.equal(dw, 1.0 + want[2])
    only = torch.ones(300, device=DEV)
    out = rl.linear_cross_entropy(*args, need_weight=False, grad_bias=only)
    assert out[2] is None and torch.equal(only, db)


@gpu
def test_gradients_against_differences():
    """Central differences of the float64 loss, step 1e-5 (their own error is below 1e-8): what is left is the
    gradients' tolerance as above."""
    c = make(6, 16, 30, "fp16", ignored=0.2, seed=4)
    _, out = run_case(c, z_loss=0.05)
    want = expected(c, 0.05)
    for k, g in (("h", out[1]), ("w", out[2]), ("b", out[3])):
        base = c[k]
        diff = torch.zeros(base.shape, dtype=torch.float64)
        for j in range(base.numel()):
            ends = []
            for sign in (1, -1):
                t = base.double().clone()
                t.view(-1)[j] += sign * 1e-5
                ends.append(loss64({**c, k: t}, 0.05))
            diff.view(-1)[j] = (ends[0] - ends[1]) / 2e-5
        name = {"h": "grad_hidden", "w": "grad_weight", "b": "grad_bias"}[k]
        check(name, g, (diff, want[name][1] + 1e-8), U["fp16"], SUB["fp16"])


def loss64(c, z_loss):
    keep = c["y"] != IGNORE
    z = c["h"].double()[keep] @ c["w"].double().t() + c["b"].double()
    lse = torch.logsumexp(z, 1)
    return (lse - z.gather(1, c["y"][keep][:, None])[:, 0] + z_loss * lse ** 2).mean()


@gpu
def test_agrees_with_the_selective_log_probabilities():
    """Without a penalty the loss is minus the mean log-probability of the targets (both within their tolerances)."""
    c = make(500, 256, 3000, seed=8)
    args = on_device(c)
    logp, _ = rl.selective_logprob_fwd(*args)
    want = expected(c)["loss"]
    assert abs(float(-logp.double().mean()) - float(rl.linear_cross_entropy_fwd(*args))) <= 2 * float(want[1])


@gpu
def test_autograd():
    c = make(60, 64, 300, ignored=0.3)
    args = on_device(c)
    h, w, b = (t.clone().requires_grad_() for t in args[:3])
    loss = rl.linear_cross_entropy_autograd(h, w, b, args[3], z_loss=1e-3)
    (3.0 * loss).backward()
    want = rl.linear_cross_entropy(*args, z_loss=1e-3)
    assert torch.equal(loss.detach(), want[0])
    for t, g in zip((h, w, b), want[1:]):
        assert torch.equal(t.grad, (g.float() * 3.0).to(g.dtype))
    h2 = args[0].clone().requires_grad_()
    rl.linear_cross_entropy_autograd(h2, args[1], args[2], args[3], z_loss=1e-3).backward()
    assert torch.equal(h2.grad, want[1])
    with torch.no_grad():
        assert torch.equal(rl.linear_cross_entropy_autograd(h, w, b, args[3], z_loss=1e-3), want[0])
    compiled = torch.compile(lambda x: rl.linear_cross_entropy_autograd(x, args[1], args[2], args[3], z_loss=1e-3),
                             fullgraph=True, backend="aot_eager")
    h3 = args[0].clone().requires_grad_()
    compiled(h3).backward()
    assert torch.equal(h3.grad, want[1])


@gpu
def test_graph_replays():
    n, H, V = 300, 64, 1000
    sets = [make(n, H, V, ignored=0.3, seed=s) for s in range(4)]
    static = on_device(sets[0])
    ws = torch.empty(rl.library().linear_cross_entropy_workspace_bytes(n, H, V, 1) + 256, dtype=torch.uint8, device=DEV)
    call = lambda w: rl.linear_cross_entropy(*static, z_loss=1e-3, workspace=w)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(ws)
    for c in sets[1:]:
        for t, new in zip(static, on_device(c)):
            t.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = call(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@gpu
def test_two_streams_at_once():
    c = [on_device(make(500, 128, 4000, seed=s)) for s in range(2)]
    want = [rl.linear_cross_entropy(*a) for a in c]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append([])
        for s, a in zip(streams, c):
            with torch.cuda.stream(s):
                got[-1].append(rl.linear_cross_entropy(*a))
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


@gpu
def test_full_size_sampled():
    """1024 x 4096 x 128256 with targets that count in four rows only: every gradient comes from those rows."""
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    h, w = r(1024, 4096).bfloat16(), (r(128256, 4096) * 2 / 64).bfloat16()
    b = (0.5 * r(128256)).bfloat16()
    y = torch.full((1024,), IGNORE, device=DEV)
    rows = torch.tensor([0, 333, 777, 1023], device=DEV)
    y[rows] = torch.tensor([0, 128255, 77777, 256], device=DEV)
    loss, dh, dw, db = rl.linear_cross_entropy(h, w, b, y)
    c = {"h": h[rows].cpu(), "w": w.cpu(), "b": b.cpu(), "y": y[rows].cpu()}
    want = expected(c)
    check("loss", loss, want["loss"])
    check("grad_hidden", dh[rows], want["grad_hidden"], U["bf16"])
    check("grad_weight", dw, want["grad_weight"], U["bf16"])
    check("grad_bias", db, want["grad_bias"], U["bf16"])
    dh[rows] = 0
    assert not dh.any()


# ------------------------------------------------------------------------------------------------------- refusals

A = 0x7F0000001000
WS = 0x7F0000100000


def call(grads, **over):
    a = dict(h=A, w=A + 0x100000, b=A + 0x200000, y=A + 0x300000, n=64, H=256, V=1000, dtype=2, ignore=-100, z=0.0, red=0,
             loss=A + 0x400000, dh=A + 0x500000, dw=A + 0x600000, db=A + 0x700000, wdt=2, acc=0, ws=WS, nbytes=64 << 20)
    a.update(over)
    common = [a["h"], a["w"], a["b"], a["y"], a["n"], a["H"], a["V"], a["dtype"], a["ignore"], ctypes.c_float(a["z"]),
              a["red"], a["loss"]]
    lib = rl.library()
    if grads:
        return rl.STATUS[lib.linear_cross_entropy(*common, a["dh"], a["dw"], a["db"], a["wdt"], a["acc"], a["ws"],
                                                  a["nbytes"], None)]
    return rl.STATUS[lib.linear_cross_entropy_fwd(*common, a["ws"], a["nbytes"], None)]


def test_refusals_of_the_c_entry_points():
    for want, over in [("RLPL_ERR_NULL", dict(h=None)), ("RLPL_ERR_NULL", dict(w=None)), ("RLPL_ERR_NULL", dict(y=None)),
                       ("RLPL_ERR_NULL", dict(loss=None)), ("RLPL_ERR_SHAPE", dict(n=0)),
                       ("RLPL_ERR_SHAPE", dict(n=(1 << 24) + 1)), ("RLPL_ERR_SHAPE", dict(H=12)),
                       ("RLPL_ERR_SHAPE", dict(H=0)), ("RLPL_ERR_SHAPE", dict(H=65544)), ("RLPL_ERR_SHAPE", dict(V=0)),
                       ("RLPL_ERR_SHAPE", dict(V=1 << 22)), ("RLPL_ERR_SHAPE", dict(n=1 << 24, V=1 << 20)),
                       ("RLPL_ERR_DTYPE", dict(dtype=0)), ("RLPL_ERR_PARAM", dict(z=-1e-3)),
                       ("RLPL_ERR_PARAM", dict(z=2.0)), ("RLPL_ERR_PARAM", dict(z=float("nan"))),
                       ("RLPL_ERR_PARAM", dict(red=2)), ("RLPL_ERR_ALIGN", dict(h=A + 8)),
                       ("RLPL_ERR_ALIGN", dict(w=A + 0x100002)), ("RLPL_ERR_ALIGN", dict(b=A + 0x200001)),
                       ("RLPL_ERR_ALIGN", dict(y=A + 0x300004)), ("RLPL_ERR_ALIGN", dict(loss=A + 0x400002)),
                       ("RLPL_ERR_WORKSPACE", dict(ws=None)), ("RLPL_ERR_WORKSPACE", dict(nbytes=256)),
                       ("RLPL_ERR_ALIGN", dict(ws=WS + 64))]:
        assert call(True, **over) == want, over
        assert call(False, **over) == want, over
    for want, over in [("RLPL_ERR_DTYPE", dict(wdt=1)), ("RLPL_ERR_PARAM", dict(acc=1)),
                       ("RLPL_ERR_ALIGN", dict(dh=A + 0x500008)), ("RLPL_ERR_ALIGN", dict(dw=A + 0x600008)),
                       ("RLPL_ERR_ALIGN", dict(wdt=0, dw=A + 0x600004)), ("RLPL_ERR_ALIGN", dict(db=A + 0x700001))]:
        assert call(True, **over) == want, over
    size = rl.library().linear_cross_entropy_workspace_bytes
    assert size(0, 64, 100, 1) == 0 and size(8, 60, 100, 1) == 0
    # one piece of logits and dz for 1024 rows, never the logits of a long batch
    assert size(1024, 4096, 128256, 1) < 900 << 20 and size(65536, 4096, 128256, 1) < 65536 * 128256 * 2 // 4
    if not torch.cuda.is_available():
        assert call(True) == "RLPL_ERR_DEVICE" and call(False) == "RLPL_ERR_DEVICE"
        assert call(True, dh=None, dw=None, db=None, b=None) == "RLPL_ERR_DEVICE"
        assert call(True, wdt=0, acc=1, dw=A + 0x600010) == "RLPL_ERR_DEVICE"


def test_constants_match_the_header():
    import os
    import re
    from rl_post_loss_amd.training import REDUCTION
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "rl_post_loss.h")).read()
    found = dict(re.findall(r"RLPL_REDUCE_(\w+) = (\d)", text))
    assert {k.lower(): int(v) for k, v in found.items()} == REDUCTION


def test_refusals_of_the_binding_on_the_host():
    z = torch.zeros
    with pytest.raises(TypeError):
        rl.linear_cross_entropy(z(2, 8), z(4, 8), None, z(2, dtype=torch.int64))


@gpu
def test_refusals_of_the_binding():
    h, w, b, y = on_device(make(8, 16, 40))
    bad = [(TypeError, (h.float(), w.float(), None, y), {}), (TypeError, (h, w.half(), None, y), {}),
           (ValueError, (h, w[:, :8], b, y), {}), (ValueError, (h, w, b[:5], y), {}), (ValueError, (h, w, b.half(), y), {}),
           (ValueError, (h, w, b, y.int()), {}), (ValueError, (h, w, b, y[:4]), {}), (ValueError, (h, w, b, y.cpu()), {}),
           (ValueError, (h, w, b, y), dict(reduction="none")), (rl.RlplError, (h, w, b, y), dict(z_loss=-1.0)),
           (rl.RlplError, (h[:0], w, b, y[:0]), {}), (rl.RlplError, (h[:, :12], w[:, :12], b, y), {}),
           (rl.RlplError, (h, w, b, y), dict(workspace=torch.empty(1024, dtype=torch.uint8, device=DEV)))]
    for error, args, kw in bad:
        with pytest.raises(error):
            rl.linear_cross_entropy(*args, **kw)
        with pytest.raises(error):
            rl.linear_cross_entropy_fwd(*args, **kw)
    f = torch.zeros(40, 16, device=DEV)
    for error, kw in [(TypeError, dict(weight_grad_dtype=torch.float16)), (ValueError, dict(grad_weight=f)),
                      (ValueError, dict(grad_weight=f.bfloat16(), grad_bias=f[:, 0].contiguous())),
                      (ValueError, dict(grad_weight=f[:8], grad_bias=torch.zeros(40, device=DEV))),
                      (ValueError, dict(grad_weight=f, grad_bias=torch.zeros(40, device=DEV),
                                        weight_grad_dtype=torch.bfloat16))]:
        with pytest.raises(error):
            rl.linear_cross_entropy(h, w, b, y, **kw)
