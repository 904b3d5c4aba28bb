"""RMS norm with the residual's addition, in the input's type and in 8 bits, and its backward pass, against float64.

Tolerances (per element, evaluated in float64 from what the kernel read; eps = 2^-24, the most a float32 operation is off
relative to its result; u = half a step of the output type, torch.finfo(t).eps / 2, plus 2^-25 below fp16's normals):

* h is one float32 addition, rounded to the stream's type: equal to torch's.
* The mean square is a sum of positive terms, a lane's 16 to 32 one after the other, then a tree of at most 10 levels and
  16 wavefronts: (32 + 26 + 2) eps; rstd = 1 / sqrt(. + norm's eps) relative by half of that and 3 eps: 33 eps.
* y = h rstd w by 33 + 2 eps, and u |y|.
* 8 bits: scale = top / 448 by 35 + 2 eps; a = y / scale = y (448 / top) off by 2 * 35 + 3 eps, and the value that holds it
  by half a step of e4m3 there: 2^(e - 4) for 2^e <= |a|, 2^-10 under 2^-6.
* Backward (rstd is an input, exact): xhat by eps; c = avg(g xhat) by (H / 64 + 35) eps of the average magnitude, as a
  wavefront takes a row in H / 64 steps at most; dh by rstd (5 eps (|g| + |xhat c|) + |xhat| e_c) + eps |dh| + u |dh|;
  dw by (n + 40) eps sum |dy xhat| + u |dw|.
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


def check(name, got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off; worst {(got - want).abs()[bad].max():.3e}, " \
                          f"allowed there {tol.expand_as(want)[bad].min():.3e}"


def make(n, H, dtype, residual="none", wdtype=None, seed=0):
    g = torch.Generator().manual_seed(seed + 131 * n + H)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rt = None if residual == "none" else torch.float32 if residual == "fp32" else DT[dtype]
    return {"x": r(n, H).to(DT[dtype]), "w": (1 + 0.2 * r(H)).to(DT[wdtype or dtype]),
            "residual": None if rt is None else (2 * r(n, H)).to(rt), "dy": r(n, H).to(DT[dtype]),
            "dstream": None if rt is None else r(n, H).to(rt)}


def dev(t):
    return None if t is None else t.to(DEV)


def stream_of(x, residual):
    return x if residual is None else (x.float() + residual.float()).to(residual.dtype)


def half_step(a):
    """Half of the distance between the e4m3 values around |a|."""
    return torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 4)


def forward_case(x, w, residual, eps, rstd, stream, y=None, q=None, scale=None):
    h = stream_of(x, residual)
    assert (stream is None) == (residual is None)
    if residual is not None:
        assert stream.dtype == residual.dtype and torch.equal(stream.cpu(), h)
    hd = h.double()
    r = 1.0 / (hd.square().mean(-1, keepdim=True) + eps).sqrt()
    check("rstd", rstd, r[..., 0], 33 * E32 * r[..., 0])
    want = hd * r * (1.0 if w is None else w.double())
    if y is not None:
        assert y.dtype == x.dtype
        check("y", y, want, 35 * E32 * want.abs() + rounding(want, y.dtype))
    if q is not None:
        assert q.dtype == torch.float8_e4m3fn and scale.dtype == torch.float32
        H = x.shape[-1]
        pad = torch.nn.functional.pad(want, (0, -H % 128))
        top = pad.unflatten(-1, (-1, 128)).abs().amax(-1)
        check("scale", scale, top / 448, 37 * E32 * top / 448)
        wide = (top / 448).repeat_interleave(128, dim=-1)[..., :H]
        a = torch.where(wide > 0, want / wide, 0.0)
        slack = 73 * E32 * a.abs()
        check("q", q.float(), a, half_step(a.abs() + slack) + slack)


SHAPES = [(1, 1), (1, 4096), (3, 2), (5, 7), (4, 64), (9, 128), (7, 129), (33, 512), (9, 513), (130, 1024), (7, 2048),
          (6, 2056), (257, 96), (3, 4100), (5, 8192), (2, 8199), (2, 16384), (3, 12345), (300, 130), (1500, 40), (40, 15),
          (25, 256), (90, 250), (7, 264), (2, 6144), (3, 6145), (4, 7000)]


@gpu
@pytest.mark.parametrize("dtype,residual", [("bf16", "none"), ("bf16", "same"), ("bf16", "fp32"), ("fp16", "same"),
                                            ("fp16", "fp32"), ("fp32", "none"), ("fp32", "same")])
@pytest.mark.parametrize("n,H", SHAPES)
def test_against_float64(n, H, dtype, residual):
    c = make(n, H, dtype, residual)
    d = {k: dev(t) for k, t in c.items()}
    y, rstd, h = rl.rms_norm_fwd(d["x"], d["w"], d["residual"], eps=1e-5)
    forward_case(c["x"], c["w"], c["residual"], 1e-5, rstd, h, y=y)
    q, scale, rstd8, h8 = rl.rms_norm_fp8(d["x"], d["w"], d["residual"], eps=1e-5)
    assert torch.equal(rstd8, rstd) and (h is None or torch.equal(h8, h))
    forward_case(c["x"], c["w"], c["residual"], 1e-5, rstd8, h8, q=q, scale=scale)
    h = d["x"] if h is None else h
    dh, dw = rl.rms_norm_bwd(d["dy"], h, d["w"], rstd, d["dstream"])
    backward_case(c["dy"], h.cpu(), c["w"], rstd.cpu(), c["dstream"], dh, dw)


def backward_case(dy, h, w, rstd, dstream, dh, dw):
    n, H = h.numel() // h.shape[-1], h.shape[-1]
    r = rstd.double()[..., None]
    xh = h.double() * r
    d = dy.double()
    g = d * (1.0 if w is None else w.double())
    c = (g * xh).mean(-1, keepdim=True)
    if dh is not None:
        e_c = (H / 64 + 36) * E32 * (g * xh).abs().mean(-1, keepdim=True)
        want = r * (g - xh * c) + (0.0 if dstream is None else dstream.double())
        assert dh.dtype == h.dtype
        check("grad_h", dh, want, (r * (5 * E32 * (g.abs() + (xh * c).abs()) + xh.abs() * e_c) + E32 * want.abs()) * 1.01
              + rounding(want, dh.dtype))
    if dw is not None:
        assert dw.dtype == w.dtype
        flat = (d * xh).reshape(n, H)
        check("grad_weight", dw, flat.sum(0), (n + 40) * E32 * flat.abs().sum(0) + rounding(flat.sum(0), dw.dtype))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_float32_weight_no_weight_and_unwanted_gradients(dtype):
    c = make(70, 264, dtype, "same", "fp32")
    d = {k: dev(t) for k, t in c.items()}
    y, rstd, h = rl.rms_norm_fwd(d["x"], d["w"], d["residual"])
    forward_case(c["x"], c["w"], c["residual"], 1e-6, rstd, h, y=y)
    full = rl.rms_norm_bwd(d["dy"], h, d["w"], rstd, d["dstream"])
    backward_case(c["dy"], h.cpu(), c["w"], rstd.cpu(), c["dstream"], *full)
    no_stream = rl.rms_norm_bwd(d["dy"], h, d["w"], rstd)
    backward_case(c["dy"], h.cpu(), c["w"], rstd.cpu(), None, *no_stream)
    dh, none = rl.rms_norm_bwd(d["dy"], h, d["w"], rstd, d["dstream"], need_weight=False)
    assert none is None and torch.equal(dh, full[0])
    none, dw = rl.rms_norm_bwd(d["dy"], h, d["w"], rstd, d["dstream"], need_h=False)
    assert none is None and torch.equal(dw, full[1])
    y, rstd, _ = rl.rms_norm_fwd(d["x"])
    forward_case(c["x"], None, None, 1e-6, rstd, None, y=y)
    dh, none = rl.rms_norm_bwd(d["dy"], d["x"], None, rstd)
    assert none is None
    backward_case(c["dy"], c["x"], None, rstd.cpu(), None, dh, None)


@gpu
def test_leading_dimensions_strides_and_unaligned_rows():
    c = make(60, 203, "bf16", "same", seed=5)
    d = {k: dev(t) for k, t in c.items()}
    x = torch.cat([d["x"], d["x"]], 1)[:, 203:]            # strided, and off 16 bytes
    y, rstd, h = rl.rms_norm_fwd(x.view(3, 20, 203) if x.is_contiguous() else x.unflatten(0, (3, 20)), d["w"],
                                 d["residual"].view(3, 20, 203))
    assert y.shape == h.shape == (3, 20, 203) and rstd.shape == (3, 20)
    ref = rl.rms_norm_fwd(d["x"], d["w"], d["residual"])
    assert torch.equal(y.view(60, 203), ref[0]) and torch.equal(h.view(60, 203), ref[2])
    flat = torch.empty(1 + 60 * 203, dtype=torch.bfloat16, device=DEV)
    flat[1:] = d["x"].view(-1)
    off = flat[1:].view(60, 203)
    assert off.data_ptr() % 16 != 0
    assert torch.equal(rl.rms_norm_fwd(off, d["w"], d["residual"])[0], ref[0])
    q, scale, _, _ = rl.rms_norm_fp8(off.view(3, 4, 5, 203), d["w"])
    assert q.shape == (3, 4, 5, 203) and scale.shape == (3, 4, 5, 2)


@gpu
@pytest.mark.parametrize("H", [5, 96, 1001, 4096, 8199])
def test_stream_written_over_the_residual(H):
    """The C entry lets h take the residual's place."""
    c = make(37, H, "bf16", "fp32")
    d = {k: dev(t) for k, t in c.items()}
    y, rstd, h = rl.rms_norm_fwd(d["x"], d["w"], d["residual"])
    out, rs = torch.empty_like(y), torch.empty_like(rstd)
    r = d["residual"].clone()
    assert rl.library().rms_norm_fwd(d["x"].data_ptr(), d["w"].data_ptr(), r.data_ptr(), 37, H, 2, 2, 0, 1e-6, out.data_ptr(),
                                     rs.data_ptr(), r.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(r, h) and torch.equal(out, y) and torch.equal(rs, rstd)


@gpu
def test_rows_of_zeros_infinities_and_nan():
    x = torch.randn(6, 300).bfloat16()
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 200] = float("nan")
    x[4, :128] = 0                                        # a group of zeros beside others
    x[5] = 1e-38                                          # squares that float32 loses
    y, rstd, _ = rl.rms_norm_fwd(x.to(DEV), eps=1e-6)
    q, scale, _, _ = rl.rms_norm_fp8(x.to(DEV), eps=1e-6)
    y, q, scale = y.float().cpu(), q.float().cpu(), scale.cpu()
    ok = [0, 1, 4, 5]
    forward_case(x[ok], None, None, 1e-6, rstd[ok], None, q=q[ok].to(torch.float8_e4m3fn), scale=scale[ok])
    assert (y[1] == 0).all() and (q[1] == 0).all() and (scale[1] == 0).all()
    assert rstd[2] == 0 and y[2, 7].isnan() and (y[2, [0, 6, 8, 299]] == 0).all()
    assert q[2, 7].isnan() and (q[2, [0, 6, 8, 299]] == 0).all() and (scale[2] == 0).all()
    assert y[3].isnan().all() and q[3].isnan().all()
    assert scale[4, 0] == 0 and scale[4, 1] > 0
    zero, rstd, _ = rl.rms_norm_fwd(torch.zeros(2, 64, device=DEV), eps=0.0)
    assert rstd.isinf().all() and zero.isnan().all()      # 0 / 0


def formula(x, w, residual, eps):
    h = x if residual is None else x + residual
    return h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * w, h


@gpu
@pytest.mark.parametrize("residual", ["none", "same"])
def test_autograd_against_torch_and_differences(residual):
    c = make(23, 77, "fp32", residual)
    leaves = [t for t in (c["x"], c["w"], c["residual"]) if t is not None]
    mine = [t.to(DEV).requires_grad_() for t in leaves]
    out = rl.rms_norm_autograd(mine[0], mine[1], mine[2] if len(mine) > 2 else None, eps=1e-5)
    y, h = out if residual != "none" else (out, None)
    loss = (y * c["dy"].to(DEV)).sum() + (0 if h is None else (h * c["dstream"].to(DEV)).sum())
    loss.backward()
    wide = [t.double().requires_grad_() for t in leaves]

    def f(ts):
        y, h = formula(ts[0], ts[1], ts[2] if len(ts) > 2 else None, 1e-5)
        return (y * c["dy"].double()).sum() + (0 if c["dstream"] is None else (h * c["dstream"].double()).sum())

    f(wide).backward()
    g = torch.Generator().manual_seed(1)
    for a, b in zip(mine, wide):
        # a hundred float32 steps of terms up to the largest gradient
        assert ((a.grad.cpu().double() - b.grad).abs() <= 200 * E32 * b.grad.abs().max().clamp(min=1)).all()
        # central differences in float64 along a direction: the error of order t^2 and of rounding are both below 1e-6
        v, t = torch.randn(b.shape, generator=g, dtype=torch.float64), 1e-5
        at = lambda s: f([w.detach() + (s * v if w is b else 0) for w in wide])  # noqa: E731,B023
        diff = (at(t) - at(-t)) / (2 * t)
        got = (a.grad.cpu().double() * v).sum()
        assert abs(got - diff) <= 1e-6 * (1 + (a.grad.cpu().double() * v).abs().sum())


@gpu
def test_autograd_mixed_types_and_single_gradients():
    c = make(12, 96, "bf16", "fp32")
    x, w, r = (c[k].to(DEV).requires_grad_() for k in ("x", "w", "residual"))
    y, h = rl.rms_norm_autograd(x, w, r)
    assert y.dtype == torch.bfloat16 and h.dtype == torch.float32
    (h * c["dstream"].to(DEV)).sum().backward()            # only the stream is used
    assert torch.equal(r.grad, c["dstream"].to(DEV)) and torch.equal(x.grad, c["dstream"].bfloat16().to(DEV)) and w.grad is None
    y, h = rl.rms_norm_autograd(x.detach(), w, r.detach())
    y.backward(c["dy"].to(DEV))
    _, rstd, hh = rl.rms_norm_fwd(x, w, r)
    assert torch.equal(w.grad, rl.rms_norm_bwd(c["dy"].to(DEV), hh, w, rstd)[1])
    traced = torch.compile(lambda a: rl.rms_norm_autograd(a, w.detach(), r.detach())[0], fullgraph=True, backend="aot_eager")
    assert torch.equal(traced(x.detach()), y)


@gpu
def test_another_stream_and_a_replayed_graph():
    c = make(50, 520, "bf16", "same")
    d = {k: dev(t) for k, t in c.items()}
    ref = rl.rms_norm_fp8(d["x"], d["w"], d["residual"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = rl.rms_norm_fp8(d["x"], d["w"], d["residual"])
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rl.rms_norm_fp8(d["x"], d["w"], d["residual"])
        grads = rl.rms_norm_bwd(d["dy"], out[3], d["w"], out[2], d["dstream"])
    for i in range(3):
        d["x"].copy_(torch.randn(50, 520, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        ref = rl.rms_norm_fp8(d["x"], d["w"], d["residual"])
        back = rl.rms_norm_bwd(d["dy"], ref[3], d["w"], ref[2], d["dstream"])
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*out, *grads), (*ref, *back)))


@gpu
def test_past_32_bits_of_elements():
    n, H = (2 ** 31) // 8192 + 3, 8192
    x = torch.zeros(n, H, dtype=torch.float16, device=DEV)
    tail = torch.randn(3, H, generator=torch.Generator().manual_seed(2)).half()
    x[-3:] = tail.to(DEV)
    w = torch.ones(H, dtype=torch.float16, device=DEV)
    y, rstd, _ = rl.rms_norm_fwd(x, w)
    forward_case(tail, w.cpu(), None, 1e-6, rstd[-3:], None, y=y[-3:])
    dh, dw = rl.rms_norm_bwd(x, x, w, rstd)
    backward_case(tail, tail, None, rstd[-3:].cpu(), None, dh[-3:], None)
    del y, dh
    q, scale, _, _ = rl.rms_norm_fp8(x, w)
    forward_case(tail, w.cpu(), None, 1e-6, rstd[-3:], None, q=q[-3:], scale=scale[-3:])


@gpu
def test_refusals_of_tensors():
    x, w = torch.zeros(4, 8, device=DEV), torch.ones(8, device=DEV)
    for bad, error in [((x.cpu(), w), TypeError), ((x.int(), w), TypeError), ((x, w.half()), TypeError),
                       ((x, w[:4]), ValueError), ((x, w, x.half()), TypeError), ((x, w, x[:2]), ValueError),
                       ((x[:0], w), rl.RlplError), ((torch.zeros(2, 16385, device=DEV),), rl.RlplError)]:
        for f in (rl.rms_norm_fwd, rl.rms_norm_fp8):
            with pytest.raises(error):
                f(*bad)
    rstd = torch.ones(4, device=DEV)
    for bad, error in [((x, x.half(), w, rstd), ValueError), ((x, x, w, rstd[:2]), ValueError), ((x, x, w, rstd, x.half()), ValueError),
                       ((x, x[:2], w, rstd), ValueError), ((x.cpu(), x, w, rstd), TypeError)]:
        with pytest.raises(error):
            rl.rms_norm_bwd(*bad)
    with pytest.raises(rl.RlplError):
        rl.rms_norm_bwd(x, x, w, rstd, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_refusals_of_the_c_entries():
    lib = rl.library()
    P = ctypes.c_void_p(0x7F0000000000)
    fwd = lambda **k: lib.rms_norm_fwd(*(k.get(n, v) for n, v in dict(  # noqa: E731
        x=P, w=P, r=None, rows=4, cols=8, dt=2, wdt=2, sdt=2, eps=1e-6, y=P, rstd=None, s=None, stream=None).items()))
    fp8 = lambda **k: lib.rms_norm_fp8(*(k.get(n, v) for n, v in dict(  # noqa: E731
        x=P, w=P, r=None, rows=4, cols=8, dt=2, wdt=2, sdt=2, eps=1e-6, q=P, scale=P, rstd=None, s=None, stream=None).items()))
    bwd = lambda **k: lib.rms_norm_bwd(*(k.get(n, v) for n, v in dict(  # noqa: E731
        gy=P, h=P, w=P, rstd=P, gs=None, rows=4, cols=8, dt=2, wdt=2, sdt=2, gh=P, gw=P, ws=P, wn=1 << 30, stream=None).items()))
    odd = ctypes.c_void_p(0x7F0000000001)
    for f in (fwd, fp8, bwd):
        assert f() == 7 or torch.cuda.is_available()       # valid: the device is asked for next
        for rows in (0, -1, 1 << 31):
            assert f(rows=rows) == 2
        for cols in (0, -8, 16385):
            assert f(cols=cols) == 2
        assert f(dt=3) == 4 and f(wdt=1) == 4 and f(sdt=1) == 4
        assert f(w=odd) == 3
    for f in (fwd, fp8):
        assert f(x=None) == 1 and f(r=P) == 1 and f(eps=float("nan")) == 5 and f(eps=-1.0) == 5 and f(x=odd) == 3
        assert f(r=P, s=odd) == 3
    assert fwd(y=None) == 1 and fp8(q=None) == 1 and fp8(scale=None) == 1 and fwd(y=odd) == 3
    assert bwd(gy=None) == 1 and bwd(h=None) == 1 and bwd(rstd=None) == 1 and bwd(ws=None) == 6 and bwd(wn=16) == 6
    assert bwd(ws=ctypes.c_void_p(0x7F0000000010)) == 3 and bwd(gh=odd) == 3 and bwd(gs=odd) == 3
    assert lib.rms_norm_workspace_bytes(4, 8) > 0 and lib.rms_norm_workspace_bytes(0, 8) == 0
    assert lib.rms_norm_workspace_bytes(4, 16385) == 0
