"""Products of 8-bit operands with scales, against float64, and the quantisation of those operands.

Tolerances (eps = 2^-24): products of two e4m3 values are exact.  float32 outputs sum them in float32 in an order and with an
intermediate rounding of the matrix core's own, which may be towards zero: 128 * 2 eps of a block's magnitudes.  16-bit
outputs sum each aligned eight of them after dropping what lies below 2^-13 of the largest, so each of the other seven
is off by 2^-13 of it at most (products of 256 * 256 and 1 * 4, 12 and 30 in one group of eight give 65536 + 0, 8 and 24;
in two groups all of it), and the groups in float32 as above.  Blocks are scaled (3 eps) and added one after the other or in
shares, and the bias: (2 * 128 + H / 128 + 8) eps sum |x w| s + eps |out|, with 16 bits 7 * 2^-13 sum over the groups of
max |x w| s more, and half a step of the output.  Quantisation is a few IEEE float32 operations: equal to torch's, bit for bit.
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


def quantised(x, rows):
    """fp8_quantize on the host."""
    R, C = x.shape
    r, c = -(-R // rows), -(-C // 128)
    a = torch.nn.functional.pad(x.float(), (0, c * 128 - C, 0, r * rows - R)).view(r, rows, c, 128)
    finite = a.isfinite()
    top = torch.where(finite, a.abs(), 0.0).amax(dim=(1, 3))
    live = top >= 2.0 ** -118
    scale = torch.where(live, top * torch.tensor(1 / 448.0), 0.0)
    inv = torch.where(live, torch.full_like(top, 448.0) / top, 0.0)   # a number over a tensor would be a reciprocal times it
    q = (a * inv[:, None, :, None])
    q = torch.where(finite, q.clamp(-448, 448), math.nan).view(r * rows, c * 128)[:R, :C]
    return q.to(torch.float8_e4m3fn), scale


def wide(q, scale, rows):
    return q.double() * scale.double().repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def make(n, H, V, seed=0):
    g = torch.Generator().manual_seed(seed + n + 3 * H + 5 * V)
    x = torch.randn(n, H, generator=g) * torch.exp(torch.randn(n, 1, generator=g))
    w = torch.randn(V, H, generator=g) * 2 / H ** 0.5
    return *quantised(x, 1), *quantised(w, 128), torch.randn(V, generator=g)


def dropped(a, b):
    """7 * 2^-13 of the largest product of each aligned eight, summed over them."""
    total = torch.zeros(a.shape[0], b.shape[0])
    for k in range(0, a.shape[1], 8):
        x, y = a[:, k:k + 8].abs().float(), b[:, k:k + 8].abs().float()
        top = torch.zeros_like(total)
        for i in range(x.shape[1]):
            top = torch.maximum(top, x[:, i:i + 1] * y[:, i])
        total += top
    return 7.01 * 2.0 ** -13 * total.double()


def product_case(x, xs, w, ws, bias, out, block_rows=128):
    a, b = wide(x, xs, 1), wide(w, ws, block_rows)
    want = a @ b.t()
    tol = (256 + x.shape[1] / 128 + 8) * E32 * (a.abs() @ b.abs().t())
    if out.dtype != torch.float32:
        tol = tol + dropped(a, b)
    if bias is not None:
        want = want + bias.double()
        tol = tol + E32 * want.abs()
    got = out.cpu().double()
    half = torch.finfo(out.dtype).eps / 2 * want.abs() + (2.0 ** -25 if out.dtype == torch.float16 else 0.0)
    bad = ~((got - want).abs() <= tol * 1.01 + half)
    assert got.shape == want.shape and not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


SHAPES = [(1, 16, 1), (1, 128, 16), (1, 4096, 300), (2, 144, 65), (16, 256, 64), (17, 512, 129), (33, 272, 700), (64, 1024, 1000),
          (65, 384, 257), (100, 1040, 515), (128, 128, 256), (129, 2048, 384), (256, 512, 512), (257, 640, 513), (300, 4096, 1003),
          (700, 256, 2051), (1, 65536, 40), (1000, 80, 90), (20, 1152, 70), (40, 2176, 130), (33, 2064, 64), (65, 8208, 129)]


@gpu
@pytest.mark.parametrize("n,H,V", SHAPES)
def test_against_float64(n, H, V):
    x, xs, w, ws, b = make(n, H, V)
    d = [t.to(DEV) for t in (x, xs, w, ws)]
    for i, (name, dtype) in enumerate(DT.items()):
        bias = b.to(dtype) if (n + i) % 2 else None
        out = rl.fp8_linear(*d, None if bias is None else bias.to(DEV), out_dtype=dtype)
        assert out.dtype == dtype
        product_case(x, xs, w, ws, bias, out)


@gpu
@pytest.mark.parametrize("n,H,V", [(700, 2064, 40001), (1100, 144, 12001), (1500, 400, 30011), (257, 8192, 33000),
                                   (128, 2064, 50001), (65, 1040, 70003), (410, 1616, 7781)])
def test_larger_tiles_by_some_of_their_results(n, H, V):
    """Sizes that take the tiles of 256, of 128 and of 128 x 64, at rows and columns around the tiles' ends and some others."""
    x, xs, w, ws, b = make(n, H, V)
    rows = torch.tensor(sorted({r for r in (0, 1, 15, 16, 63, 64, 127, 128, 255, 256, 257, n // 2, n - 65, n - 2, n - 1) if r < n}))
    g = torch.Generator().manual_seed(0)
    cols = torch.unique(torch.cat([torch.arange(300), torch.arange(V - 300, V), torch.randint(0, V, (500,), generator=g)]))
    scales = ws.repeat_interleave(128, 0)[cols]
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        bias = b.to(dtype)
        out = rl.fp8_linear(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), bias.to(DEV), out_dtype=dtype).cpu()
        pick = w.view(torch.uint8)[cols].view(torch.float8_e4m3fn)
        product_case(x.view(torch.uint8)[rows].view(torch.float8_e4m3fn), xs[rows], pick, scales, bias[cols], out[rows][:, cols], 1)


@gpu
def test_small_integers_are_exact():
    """Which element meets which: products of small integers with scales of powers of two have no rounding."""
    g = torch.Generator().manual_seed(1)
    for n, H, V in ((5, 272, 200), (300, 528, 300), (1100, 144, 12001), (700, 2064, 40001)):
        x, w = (torch.randint(-3, 4, s, generator=g).float() for s in ((n, H), (V, H)))
        xs = torch.exp2(torch.randint(-2, 2, (n, -(-H // 128)), generator=g).float())
        ws = torch.exp2(torch.randint(-2, 2, (-(-V // 128), -(-H // 128)), generator=g).float())
        q, p = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
        d = [t.to(DEV) for t in (q, xs, p, ws)]
        want = wide(d[0], d[1], 1) @ wide(d[2], d[3], 128).t()
        assert torch.equal(rl.fp8_linear(*d, out_dtype=torch.float32).double(), want)
        for dtype in (torch.bfloat16, torch.float16):      # |sums| stay in fp16's range; one rounding
            assert torch.equal(rl.fp8_linear(*d, out_dtype=dtype), want.to(dtype))


@gpu
def test_leading_dimensions_strides_and_alignment():
    x, xs, w, ws, b = make(12, 160, 333)
    d = [t.to(DEV) for t in (x, xs, w, ws)]
    ref = rl.fp8_linear(*d)
    assert torch.equal(rl.fp8_linear(d[0].view(3, 4, 160), d[1].view(3, 4, 2), *d[2:]), ref.view(3, 4, 333))
    assert torch.equal(rl.fp8_linear(d[0][5], d[1][5], *d[2:]), rl.fp8_linear(d[0][5:6], d[1][5:6], *d[2:])[0])
    flat = torch.empty(3 + 12 * 160, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    flat[3:] = d[0].reshape(-1)
    assert torch.equal(rl.fp8_linear(flat[3:].view(12, 160), d[1], *d[2:]), ref)
    two = torch.cat([d[0].view(torch.uint8)] * 2, 1).view(torch.float8_e4m3fn)
    assert torch.equal(rl.fp8_linear(two[:, 160:], d[1].t().contiguous().t(), *d[2:]), ref)


@gpu
def test_nan_stays_in_its_row_and_column():
    for n, V in ((3, 100), (200, 300)):
        x, xs, w, ws, _ = make(n, 256, V)
        xb, wb = x.view(torch.uint8).clone(), w.view(torch.uint8).clone()
        xb[1, 200], wb[70, 3] = 0x7F, 0xFF
        out = rl.fp8_linear(xb.view(torch.float8_e4m3fn).to(DEV), xs.to(DEV), wb.view(torch.float8_e4m3fn).to(DEV), ws.to(DEV),
                            out_dtype=torch.float32).cpu()
        assert out[1].isnan().all() and out[:, 70].isnan().all()
        out[1], out[:, 70] = 0, 0
        assert out.isfinite().all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("R,C", [(1, 1), (3, 5), (1, 128), (7, 129), (128, 128), (129, 1000), (300, 513), (64, 4096), (2, 8192)])
def test_quantisation_bit_for_bit(R, C, dtype):
    g = torch.Generator().manual_seed(R + C)
    x = (torch.randn(R, C, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))).to(DT[dtype])
    x[0, 0] = 0
    if C > 200:
        x[:, 128:256] = 0
        x[R // 2, 7] = math.inf
        x[R - 1, C - 1] = math.nan
    for rows in (1, 128):
        q, scale = rl.fp8_quantize(x.to(DEV), block_rows=rows)
        want, s = quantised(x, rows)
        assert torch.equal(scale.cpu(), s)
        a, b = q.cpu().float(), want.float()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@gpu
def test_quantisation_of_views_and_tiny_values():
    x = torch.randn(40, 700, generator=torch.Generator().manual_seed(0)).to(DEV)
    for v in (x[:, 3:333], x[::3, :256], x.t()):
        for rows in (1, 128):
            q, s = rl.fp8_quantize(v, block_rows=rows)
            qq, ss = rl.fp8_quantize(v.contiguous(), block_rows=rows)
            assert torch.equal(s, ss) and torch.equal(q.view(torch.uint8), qq.view(torch.uint8))
    q, s = rl.fp8_quantize(x.view(4, 10, 700))
    assert q.shape == (4, 10, 700) and s.shape == (4, 10, 6)
    tiny = torch.full((2, 128), 2.0 ** -119, device=DEV)
    tiny[1] = 2.0 ** -118
    q, s = rl.fp8_quantize(tiny)
    assert s[0] == 0 and (q[0].float() == 0).all() and s[1] > 0 and (q[1].float() == 448).all()


@gpu
def test_another_stream_and_a_replayed_graph():
    for n, H, V in ((3, 512, 700), (300, 1024, 1500)):
        x, xs, w, ws, b = make(n, H, V)
        d = [t.to(DEV) for t in (x, xs, w, ws)]
        bias = b.bfloat16().to(DEV)
        ref = rl.fp8_linear(*d, bias)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = rl.fp8_linear(*d, bias)
        side.synchronize()
        assert torch.equal(got, ref)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = rl.fp8_linear(*d, bias)
        for i in range(3):
            d[1].mul_(1.5)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, rl.fp8_linear(*d, bias))


@gpu
def test_past_32_bits_of_output():
    n, H, V = 17000, 16, 131073
    x, xs, w, ws, _ = make(4, H, V)
    full = torch.zeros(n, H, dtype=torch.uint8, device=DEV)
    full[-4:] = x.view(torch.uint8).to(DEV)
    scales = torch.ones(n, 1, device=DEV)
    scales[-4:] = xs.to(DEV)
    out = rl.fp8_linear(full.view(torch.float8_e4m3fn), scales, w.to(DEV), ws.to(DEV))
    product_case(x, xs, w, ws, None, out[-4:])
    assert (out[-5] == 0).all() and (out[0] == 0).all()


@gpu
def test_refusals_of_tensors():
    x, xs, w, ws, b = (t.to(DEV) for t in make(4, 32, 10))
    for bad, error in [((x.float(), xs, w, ws), TypeError), ((x, xs, w.float(), ws), TypeError), ((x.cpu(), xs.cpu(), w.cpu(), ws.cpu()), TypeError),
                       ((x, xs, w[:, :16], ws), ValueError), ((x, xs[:2], w, ws), ValueError), ((x, xs.double(), w, ws), ValueError),
                       ((x, xs, w, ws.half()), ValueError), ((x, xs, w, ws, b.half()), ValueError), ((x, xs, w, ws, b[:3].bfloat16()), ValueError),
                       ((x[:0], xs[:0], w, ws), rl.RlplError)]:
        with pytest.raises(error):
            rl.fp8_linear(*bad)
    with pytest.raises(TypeError):
        rl.fp8_linear(x, xs, w, ws, out_dtype=torch.float64)
    with pytest.raises(rl.RlplError):                      # 24 columns
        rl.fp8_linear(x[:, :24], xs, w[:, :24], ws)
    with pytest.raises(rl.RlplError):
        rl.fp8_linear(x, xs, w, ws, workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
    for bad, error in [((b.int(),), TypeError), ((b.cpu(),), TypeError), ((b[:0],), rl.RlplError)]:
        with pytest.raises(error):
            rl.fp8_quantize(*bad)
    with pytest.raises(ValueError):
        rl.fp8_quantize(b, block_rows=64)
    with pytest.raises(ValueError):
        rl.fp8_quantize(b, block_rows=128)


def test_refusals_of_the_c_entries():
    lib = rl.library()
    P, odd = ctypes.c_void_p(0x7F0000000000), ctypes.c_void_p(0x7F0000000001)

    def linear(**k):
        d = dict(x=P, xs=P, w=P, ws=P, b=None, n=4, H=64, V=100, dt=2, out=P, work=P, wn=1 << 40, stream=None)
        assert set(k) <= set(d)
        return lib.fp8_linear(*(d | k).values())

    def quant(**k):
        d = dict(x=P, rows=4, cols=100, ld=100, dt=2, block=1, q=P, s=P, stream=None)
        assert set(k) <= set(d)
        return lib.rlpl_fp8_quantize(*(d | k).values())

    assert linear() == 7 and quant() == 7 and quant(block=128) == 7 or torch.cuda.is_available()
    for k in ("x", "xs", "w", "ws", "out"):
        assert linear(**{k: None}) == 1 and linear(**{k: odd}) == 3
    assert linear(b=odd) == 3 and linear(x=ctypes.c_void_p(0x7F0000000008)) == 3
    for k, bad in (("n", (0, -1, (1 << 20) + 1)), ("H", (0, 8, 24, 65552, -16)), ("V", (0, -5, 1 << 22))):
        for v in bad:
            assert linear(**{k: v}) == 2
    assert linear(dt=3) == 4 and linear(work=None) == 6 and linear(wn=1) == 6 and linear(work=ctypes.c_void_p(0x7F0000000010)) == 3
    for k in ("x", "q", "s"):
        assert quant(**{k: None}) == 1
    assert quant(rows=0) == 2 and quant(cols=0) == 2 and quant(rows=1 << 31) == 2 and quant(cols=1 << 31) == 2 and quant(ld=-1) == 2
    assert quant(ld=1 << 62) == 2 and quant(dt=7) == 4 and quant(block=2) == 5 and quant(x=odd) == 3 and quant(s=odd) == 3
    size = lib.fp8_linear_workspace_bytes
    assert size(1, 16, 1) > 0 and size(0, 16, 1) == 0 and size(1, 8, 1) == 0 and size(1, 16, 1 << 22) == 0
