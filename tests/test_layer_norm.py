"""Layer norm, forward and backward, against float64.

Tolerances (per element, evaluated in float64 from the inputs; eps = 2^-24, the most a float32 operation is off
relative to its result; u = half a step of the output type, torch.finfo(t).eps / 2, plus 2^-25 below fp16's normals):

* A float32 sum of k terms taken as s serial steps and a tree is off by at most (s + 32) eps times the sum of the
  magnitudes (two steps for each of the tree's at most 16 levels).  A lane holds at most 128 of a row's elements in
  the forward; in the backward a wavefront takes a row in H / 64 steps and a column's rows in at most n steps.
* mean: (128 + 32) eps avg|x|, so a deviation d = x - mean is off by e_d = that + eps |d|; the variance by
  2 avg|d| e_d + e_d^2 + 162 eps var; rstd relative by half the variance's error over (var + eps_norm), plus 3 eps.
* y = d rstd w + b: |w| rstd (e_d + |d| rel(rstd)) + 3 eps (|d rstd w| + |b|) + u |y|.
* Backward (mean and rstd are inputs, exact): xhat off by e_h = 2 eps |xhat| + eps |x - mean| rstd; the row averages
  c1 = avg g, c2 = avg g xhat, g = dy w (eps |g|), by (H/64 + 35) eps times the averages of the magnitudes, c2 also
  by avg(|g| e_h); dx by rstd (4 eps (|g| + |c1| + |xhat c2|) + e_c1 + |xhat| e_c2 + e_h |c2|) + u |dx|.
* dw by sum |dy| e_h + (n + 35) eps sum |dy xhat| + u |dw|, db by (n + 35) eps sum |dy| + u |db|.
"""
import ctypes

import pytest
import torch

import rl_post_loss_amd as rl

E32 = 2.0 ** -24
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
gpu = pytest.mark.gpu


def rounding(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def make(n, H, dtype, wdtype=None, affine="wb", seed=0, offset=1.0):
    g = torch.Generator().manual_seed(seed + 131 * n + H)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wdtype = wdtype or dtype
    return {"x": (1.5 * r(n, H) + offset * r(n, 1)).to(DT[dtype]),
            "w": (1 + 0.2 * r(H)).to(DT[wdtype]) if "w" in affine else None,
            "b": (0.2 * r(H)).to(DT[wdtype]) if "b" in affine else None, "dy": r(n, H).to(DT[dtype])}


def dev(t):
    return None if t is None else t.to(DEV)


def wide(t, like):
    return torch.ones_like(like[0]) if t is None else t.double()


def check(name, got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off; worst {(got - want).abs()[bad].max():.3e}, " \
                          f"allowed there {tol.expand_as(want)[bad].min():.3e}"


def forward_case(x, w, b, eps, out):
    y, mean, rstd = out
    xd = x.double()
    H = x.shape[-1]
    m = xd.mean(-1, keepdim=True)
    d = xd - m
    var = d.square().mean(-1, keepdim=True)
    r = (var + eps).rsqrt()
    e_mean = 160 * E32 * xd.abs().mean(-1, keepdim=True) + E32 * m.abs()
    e_d = e_mean + E32 * d.abs()
    e_top = e_mean + E32 * d.abs().amax(-1, keepdim=True)
    e_var = 2 * d.abs().mean(-1, keepdim=True) * e_top + e_top ** 2 + 162 * E32 * var
    rel = 0.5 * e_var / (var + eps) + 3 * E32
    wd = wide(w, xd)
    bd = torch.zeros(H, dtype=torch.float64) if b is None else b.double()
    want = d * r * wd + bd
    tol = wd.abs() * r * (e_d + d.abs() * rel) + 3 * E32 * ((d * r * wd).abs() + bd.abs())
    check("y", y, want, tol * 1.01 + rounding(want, y.dtype))
    check("mean", mean, m[..., 0], e_mean[..., 0])
    check("rstd", rstd, r[..., 0], (r * rel)[..., 0] * 1.01)


def backward_case(c, mean, rstd, out):
    x, w, dy = c["x"].double(), c["w"], c["dy"].double()
    n, H = x.shape
    m, r = mean.cpu().double()[:, None], rstd.cpu().double()[:, None]
    wd = wide(w, x)
    h = (x - m) * r
    g = dy * wd
    e_h = E32 * (2 * h.abs() + (x - m).abs() * r)
    k = (H / 64 + 35) * E32
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    e1 = k * g.abs().mean(1, keepdim=True)
    e2 = k * (g * h).abs().mean(1, keepdim=True) + (g.abs() * e_h).mean(1, keepdim=True)
    dx = r * (g - c1 - h * c2)
    tol = r * (4 * E32 * (g.abs() + c1.abs() + (h * c2).abs()) + e1 + h.abs() * e2 + e_h * c2.abs())
    kn = (n + 35) * E32
    dw, db = (dy * h).sum(0), dy.sum(0)
    if out[0] is not None:
        check("grad_x", out[0], dx, tol * 1.01 + rounding(dx, out[0].dtype))
    if out[1] is not None:
        check("grad_weight", out[1], dw, ((dy.abs() * e_h).sum(0) + kn * (dy * h).abs().sum(0)) * 1.01
              + rounding(dw, out[1].dtype))
    if out[2] is not None:
        check("grad_bias", out[2], db, kn * dy.abs().sum(0) * 1.01 + rounding(db, out[2].dtype))


SHAPES = [(1, 1), (1, 4096), (3, 2), (5, 7), (4, 64), (17, 1000), (33, 512), (9, 513), (130, 1024), (7, 2048), (6, 2056),
          (257, 96), (3, 4100), (5, 8192), (2, 16384), (2, 16385), (3, 12345), (40, 16384), (9, 12000), (300, 130), (100, 15), (40, 9000), (1, 65536), (2, 65535), (1500, 40)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,H", SHAPES)
def test_against_float64(n, H, dtype):
    c = make(n, H, dtype)
    d = {k: dev(t) for k, t in c.items()}
    out = rl.layer_norm_fwd(d["x"], d["w"], d["b"], eps=1e-5)
    forward_case(c["x"], c["w"], c["b"], 1e-5, out)
    grads = rl.layer_norm_bwd(d["dy"], d["x"], d["w"], out[1], out[2])
    assert [t.dtype for t in grads] == [DT[dtype]] * 3
    backward_case(c, out[1], out[2], grads)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("affine", ["wb", "w", "b", ""])
def test_float32_weights_and_missing_ones(dtype, affine):
    c = make(70, 264, dtype, "fp32", affine)
    d = {k: dev(t) for k, t in c.items()}
    out = rl.layer_norm_fwd(d["x"], d["w"], d["b"], eps=1e-6)
    assert out[0].dtype == DT[dtype]
    forward_case(c["x"], c["w"], c["b"], 1e-6, out)
    grads = rl.layer_norm_bwd(d["dy"], d["x"], d["w"], out[1], out[2])
    assert (grads[1] is None) == ("w" not in affine)
    if grads[1] is not None:
        assert grads[1].dtype == torch.float32 and grads[2].dtype == torch.float32
    backward_case(c, out[1], out[2], grads)


@gpu
def test_unaligned_rows_and_strided_inputs():
    """Tensors that start off 16 bytes, and views that are not contiguous, give what aligned copies give."""
    c = make(40, 256, "bf16")
    d = {k: dev(t) for k, t in c.items()}
    want = rl.layer_norm_fwd(d["x"], d["w"], d["b"])
    buf = torch.empty(40 * 256 + 1, dtype=torch.bfloat16, device=DEV)
    off = buf[1:].view(40, 256)
    off.copy_(d["x"])
    forward_case(c["x"], c["w"], c["b"], 1e-5, rl.layer_norm_fwd(off, d["w"], d["b"]))
    backward_case(c, want[1], want[2], rl.layer_norm_bwd(d["dy"], off, d["w"], want[1], want[2]))
    cols = torch.empty(40, 300, dtype=torch.bfloat16, device=DEV)[:, 20:276]
    cols.copy_(d["x"])
    assert all(torch.equal(a, b) for a, b in zip(rl.layer_norm_fwd(cols, d["w"], d["b"]), want))
    turned = d["x"].t().contiguous().t()
    assert all(torch.equal(a, b) for a, b in zip(rl.layer_norm_fwd(turned, d["w"], d["b"]), want))


@gpu
def test_rows_of_equal_values_large_offsets_and_bad_values():
    x = torch.full((3, 128), 5.0, device=DEV)
    y, mean, rstd = rl.layer_norm_fwd(x, None, None, eps=1e-5)
    assert torch.all(y == 0) and torch.all(mean == 5)
    assert torch.allclose(rstd.cpu(), torch.full((3,), (1e-5) ** -0.5), rtol=1e-6)
    c = make(20, 500, "fp32", offset=1000.0)          # deviations far below the mean
    forward_case(c["x"], c["w"], c["b"], 1e-5, rl.layer_norm_fwd(dev(c["x"]), dev(c["w"]), dev(c["b"])))
    c = make(6, 300, "bf16")
    want = rl.layer_norm_fwd(dev(c["x"]), dev(c["w"]), dev(c["b"]))[0]
    c["x"][2, 7], c["x"][4, 0] = float("nan"), float("inf")
    y = rl.layer_norm_fwd(dev(c["x"]), dev(c["w"]), dev(c["b"]))[0]
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], want[keep])           # a bad row stays in its row


@gpu
def test_leading_dimensions_wanted_gradients_and_repeats():
    c = make(60, 136, "bf16")
    d = {k: dev(t) for k, t in c.items()}
    y, mean, rstd = rl.layer_norm_fwd(d["x"].view(3, 20, 136), d["w"], d["b"])
    y1, mean1, rstd1 = rl.layer_norm_fwd(d["x"], d["w"], d["b"])
    assert y.shape == (3, 20, 136) and mean.shape == (3, 20)
    assert torch.equal(y.view(60, 136), y1) and torch.equal(mean.view(60), mean1)
    full = rl.layer_norm_bwd(d["dy"], d["x"], d["w"], mean1, rstd1)
    again = rl.layer_norm_bwd(d["dy"], d["x"], d["w"], mean1, rstd1)
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    for want in range(8):
        flags = dict(need_x=bool(want & 1), need_weight=bool(want & 2), need_bias=bool(want & 4))
        got = rl.layer_norm_bwd(d["dy"], d["x"], d["w"], mean1, rstd1, **flags)
        for g, f, need in zip(got, full, flags.values()):
            assert (g is not None) == need and (g is None or torch.equal(g, f))
    # rows after a problem's last one stay as they were
    buf = torch.full((64, 136), 7.0, dtype=torch.bfloat16, device=DEV)
    lib = rl.library()
    assert lib.layer_norm_fwd(d["x"].data_ptr(), d["w"].data_ptr(), d["b"].data_ptr(), 60, 136, 2, 2, 1e-5,
                              buf.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(buf[:60], y1) and torch.all(buf[60:] == 7)
    assert lib.layer_norm_fwd(buf.data_ptr(), d["w"].data_ptr(), d["b"].data_ptr(), 60, 136, 2, 2, 1e-5, buf.data_ptr(),
                              None, None, torch.cuda.current_stream().cuda_stream) == 0      # in place
    assert torch.equal(buf[:60], rl.layer_norm_fwd(y1, d["w"], d["b"])[0])


@gpu
@pytest.mark.parametrize("n,H", [(5, 24), (3, 17)])
def test_gradients_against_differences(n, H):
    """Central differences of sum(dy * y) in float64, step 1e-6 (error about step^2 and 1e-10): 1e-4 of the largest
    gradient leaves room for the float32 gradients' own error alone."""
    c = make(n, H, "fp32")
    d = {k: dev(t) for k, t in c.items()}
    _, mean, rstd = rl.layer_norm_fwd(d["x"], d["w"], d["b"], eps=1e-5)
    got = rl.layer_norm_bwd(d["dy"], d["x"], d["w"], mean, rstd)
    args = [c[k].double() for k in "xwb"]

    def f(x, w, b):
        return (c["dy"].double() * torch.nn.functional.layer_norm(x, (H,), w, b, 1e-5)).sum()

    for i, g in enumerate(got):
        diff = torch.zeros_like(args[i])
        for j in range(diff.numel()):
            a = [t.clone() for t in args]
            a[i].view(-1)[j] += 1e-6
            up = f(*a)
            a[i].view(-1)[j] -= 2e-6
            diff.view(-1)[j] = (up - f(*a)) / 2e-6
        assert (g.cpu().double() - diff).abs().max() <= 1e-4 * diff.abs().max()


@gpu
def test_autograd_matches_the_direct_calls():
    c = make(50, 200, "bf16")
    d = {k: dev(t) for k, t in c.items()}
    x, w, b = (d[k].clone().requires_grad_() for k in "xwb")
    y = rl.layer_norm_autograd(x, w, b, eps=1e-5)
    y.backward(d["dy"])
    y0, mean, rstd = rl.layer_norm_fwd(d["x"], d["w"], d["b"], eps=1e-5)
    want = rl.layer_norm_bwd(d["dy"], d["x"], d["w"], mean, rstd)
    assert torch.equal(y.detach(), y0)
    assert all(torch.equal(t.grad, g) for t, g in zip((x, w, b), want))
    x2 = d["x"].clone().requires_grad_()
    rl.layer_norm_autograd(x2).backward(d["dy"])      # no weight, no bias
    want = rl.layer_norm_bwd(d["dy"], d["x"], None, mean, rstd, need_bias=False)
    assert torch.equal(x2.grad, want[0]) and want[1] is None


def test_fake_implementation_gives_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        y, mean, rstd = torch.ops.rlpl.layer_norm(torch.empty(3, 5, 16, dtype=torch.bfloat16), None, None, 1e-5)
        assert y.shape == (3, 5, 16) and y.dtype == torch.bfloat16
        assert mean.shape == rstd.shape == (3, 5) and mean.dtype == torch.float32


A = 0x7F0000001000   # a fake aligned device address: refused calls never use it
WS = 0x7F0000100000


def call(backward=False, **over):
    a = dict(x=A, w=A + 0x10000, b=A + 0x20000, y=A + 0x30000, rows=8, cols=64, dtype=2, wdtype=2, eps=1e-5, mean=A + 0x40000,
             rstd=A + 0x50000, dy=A + 0x60000, dx=A + 0x70000, dw=A + 0x80000, db=A + 0x90000, ws=WS, nbytes=1 << 20)
    a.update(over)
    lib = rl.library()
    if backward:
        st = lib.layer_norm_bwd(a["dy"], a["x"], a["w"], a["mean"], a["rstd"], a["rows"], a["cols"], a["dtype"],
                                a["wdtype"], a["dx"], a["dw"], a["db"], a["ws"], a["nbytes"], None)
    else:
        st = lib.layer_norm_fwd(a["x"], a["w"], a["b"], a["rows"], a["cols"], a["dtype"], a["wdtype"],
                                ctypes.c_float(a["eps"]), a["y"], a["mean"], a["rstd"], None)
    return rl.STATUS[st]


def test_refusals_of_the_c_entry_points():
    both = [("RLPL_ERR_NULL", dict(x=None)), ("RLPL_ERR_SHAPE", dict(rows=0)), ("RLPL_ERR_SHAPE", dict(rows=1 << 31)),
            ("RLPL_ERR_SHAPE", dict(cols=0)), ("RLPL_ERR_SHAPE", dict(cols=65537)), ("RLPL_ERR_DTYPE", dict(dtype=3)),
            ("RLPL_ERR_DTYPE", dict(wdtype=1)), ("RLPL_ERR_DTYPE", dict(dtype=0, wdtype=2)),
            ("RLPL_ERR_ALIGN", dict(x=A + 1)), ("RLPL_ERR_ALIGN", dict(w=A + 0x10001)),
            ("RLPL_ERR_ALIGN", dict(mean=A + 2))]
    for want, over in both:
        assert call(**over) == want, over
        assert call(True, **over) == want, over
    for want, over in [("RLPL_ERR_NULL", dict(y=None)), ("RLPL_ERR_PARAM", dict(eps=-1.0)),
                       ("RLPL_ERR_PARAM", dict(eps=float("nan"))), ("RLPL_ERR_ALIGN", dict(b=A + 0x20001))]:
        assert call(**over) == want, over
    for want, over in [("RLPL_ERR_NULL", dict(dy=None)), ("RLPL_ERR_NULL", dict(mean=None)),
                       ("RLPL_ERR_NULL", dict(rstd=None)), ("RLPL_ERR_ALIGN", dict(dx=A + 0x70001)),
                       ("RLPL_ERR_ALIGN", dict(dw=A + 0x80001)), ("RLPL_ERR_WORKSPACE", dict(ws=None)),
                       ("RLPL_ERR_WORKSPACE", dict(nbytes=64)), ("RLPL_ERR_ALIGN", dict(ws=WS + 64))]:
        assert call(True, **over) == want, over
    assert rl.library().layer_norm_workspace_bytes(0, 64) == 0
    assert rl.library().layer_norm_workspace_bytes(8, 65537) == 0
    if not torch.cuda.is_available():
        assert call() == "RLPL_ERR_DEVICE" and call(True, w=None, dw=None) == "RLPL_ERR_DEVICE"


def test_refusals_of_the_binding_on_the_host():
    with pytest.raises(TypeError):
        rl.layer_norm_fwd(torch.zeros(2, 4))                       # not a device tensor
    with pytest.raises(TypeError):
        rl.layer_norm_bwd(torch.zeros(2, 4), torch.zeros(2, 4), None, torch.zeros(2), torch.zeros(2))


@gpu
def test_refusals_of_the_binding():
    c = {k: dev(t) for k, t in make(4, 32, "bf16").items()}
    _, mean, rstd = rl.layer_norm_fwd(c["x"], c["w"], c["b"])
    for args in ((c["x"], c["w"][:16], None), (c["x"], c["w"].cpu(), None)):
        with pytest.raises(ValueError):
            rl.layer_norm_fwd(*args)
    for args in ((c["x"].double(), None, None), (c["x"], c["w"].half(), None), (c["x"], c["w"], c["b"].float())):
        with pytest.raises(TypeError):
            rl.layer_norm_fwd(*args)
    for args in ((c["dy"][:2], c["x"], c["w"], mean, rstd), (c["dy"].float(), c["x"], c["w"], mean, rstd),
                 (c["dy"], c["x"], c["w"], mean[:2], rstd), (c["dy"], c["x"], c["w"], mean, rstd.half())):
        with pytest.raises(ValueError):
            rl.layer_norm_bwd(*args)
    with pytest.raises(rl.RlplError, match="SHAPE"):
        rl.layer_norm_fwd(torch.zeros(0, 32, device=DEV))
    with pytest.raises(rl.RlplError, match="WORKSPACE"):
        rl.layer_norm_bwd(c["dy"], c["x"], c["w"], mean, rstd, workspace=torch.empty(
            rl.library().layer_norm_workspace_bytes(4, 32) - 1, dtype=torch.uint8, device=DEV))
