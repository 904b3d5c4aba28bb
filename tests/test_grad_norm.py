"""The norm over a list of gradients, the factor that clips it, and gradients scaled in place.

Tolerances (eps = 2^-24): the sum of squares is float64 (relative error of n 2^-53 at most, n < 2^30: below 2^-23 of eps),
its root rounded to float32 once: norm by 1.01 eps (2.01 with a grad_scale, in float64 until the same rounding); scale =
max_norm / (norm + e), two float32 operations more: 4 eps with the arguments' own rounding, 5 with a grad_scale.  A scaled
element is one float32 product rounded to its type: equal to torch's.
"""
import ctypes
import math

import pytest
import torch

import rl_post_loss_amd as rl

E32 = 2.0 ** -24
DEV = "cuda:0"
gpu = pytest.mark.gpu
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def norm_of(grads, kind=2.0):
    flat = torch.cat([g.detach().double().reshape(-1).cpu() for g in grads if g is not None])
    if flat.numel() == 0:
        return 0.0
    return float(flat.abs().max() if kind == math.inf else flat.square().sum().sqrt())


def near(got, want, steps):
    got = float(got)
    assert abs(got - want) <= steps * E32 * abs(want), (got, want, abs(got - want) / abs(want) / E32)


def tensors(sizes, dtypes, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dtypes[i % len(dtypes)]).to(DEV) for i, n in enumerate(sizes)]


LISTS = {"one": [1], "small": [3, 0, 17, 4096, 1], "alone": [4096] * 16, "over alone": [4096] * 16 + [1], "empty": [0, 0],
         "full window": [5] * 190, "two windows": [7, 1000] * 96, "long": [3_000_001, 12345], "many": list(range(1, 600))}


@gpu
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("name", list(LISTS))
def test_norm_and_scale(name, kind):
    for dtypes in ([torch.float32], [torch.bfloat16], TYPES):
        grads = tensors(LISTS[name], dtypes, len(name))
        want = norm_of(grads, kind)
        near(rl.grad_norm(grads, norm_type=kind), want, 1.01)
        for max_norm in (0.5, 1e9):
            norm, scale = rl.grad_norm(grads, max_norm=max_norm, norm_type=kind, eps=1e-6)
            near(norm, want, 1.01)
            near(scale, min(1.0, max_norm / (want + 1e-6)), 4 if max_norm < want else 0)


@gpu
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_values_whose_squares_float32_does_not_hold(kind):
    for size in (1e30, 1e-30, 3e-39):                      # the last one is subnormal
        grads = [torch.full((5000,), size, device=DEV), torch.full((300, 500), -size, device=DEV)]
        near(rl.grad_norm(grads, norm_type=kind), norm_of(grads, kind), 1.01 + (2.0 ** -149 / size) / E32)
    big = [torch.full((100000,), 3e38, device=DEV)]
    assert float(rl.grad_norm(big)) == math.inf           # the norm itself is past float32
    norm, scale = rl.grad_norm(big, max_norm=1.0)
    assert float(scale) == 0.0


@gpu
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_nan_and_infinity(kind):
    for where in (0, 70000, 199999):
        for bad, want in ((math.nan, math.nan), (math.inf, math.inf), (-math.inf, math.inf)):
            grads = tensors([100000, 100000], TYPES, 3)
            grads[where // 100000][where % 100000] = bad
            norm, scale = rl.grad_norm(grads, max_norm=1.0, norm_type=kind)
            assert math.isnan(float(norm)) if math.isnan(want) else float(norm) == want
            assert math.isnan(float(scale)) if math.isnan(want) else float(scale) == 0.0
    both = torch.tensor([math.inf, math.nan, 1.0], device=DEV)
    assert math.isnan(float(rl.grad_norm([both], norm_type=kind)))


@gpu
def test_grad_scale_of_a_loss_scale():
    grads = tensors([1000, 70000, 33], [torch.float16], 5, 100.0)
    inv = torch.tensor(1.0 / 1024.0, device=DEV)
    want = norm_of(grads) / 1024
    norm, scale = rl.grad_norm(grads, max_norm=1.0, grad_scale=inv)
    near(norm, want, 2.01)
    near(scale, min(1.0, 1.0 / (want + 1e-6)) / 1024, 5)
    norm, scale = rl.grad_norm(grads, max_norm=1e6, grad_scale=inv)
    assert float(scale) == 1.0 / 1024.0
    norm, scale = rl.grad_norm(grads, max_norm=1e6, grad_scale=-inv)
    assert float(norm) > 0 and float(scale) == -1.0 / 1024.0


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_views_at_every_alignment_and_permuted_dimensions(dtype):
    flat = torch.randn(100000, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    for first in range(17):
        for n in (0, 1, 7, 15, 16, 17, 8191, 8192, 8193, 50000):
            near(rl.grad_norm([flat[first:first + n]]), norm_of([flat[first:first + n]]), 1.01)
            before = flat.clone()
            rl.scale_grads([flat[first:first + n]], torch.tensor(0.3, device=DEV))
            want = before.clone()
            want[first:first + n] = (before[first:first + n].float() * 0.3).to(dtype)
            assert torch.equal(flat, want)                 # nothing around it is written
            flat.copy_(before)
    t = flat[:60000].view(200, 300).t()
    near(rl.grad_norm([t]), norm_of([t]), 1.01)
    near(rl.grad_norm([flat[:60000].view(200, 300)[:, ::3]]), norm_of([flat[:60000].view(200, 300)[:, ::3]]), 1.01)
    near(rl.grad_norm([flat[:1].expand(50, 7)]), norm_of([flat[:1].expand(50, 7)]), 1.01)
    before = t.clone()
    rl.scale_grads([t], torch.tensor(-2.0, device=DEV))
    assert torch.equal(t, before * -2)


@gpu
@pytest.mark.parametrize("name", ["small", "alone", "two windows", "long", "many"])
def test_clipping_in_place(name):
    for dtypes in ([torch.float32], TYPES):
        grads = tensors(LISTS[name], dtypes, 11)
        before = [g.clone() for g in grads]
        norm, scale = rl.grad_norm(grads, max_norm=0.25)
        got = rl.clip_grads(grads, 0.25)
        assert torch.equal(got, norm)
        for g, b in zip(grads, before):
            assert torch.equal(g, (b.float() * scale).to(b.dtype))
        version = [g._version for g in grads]
        rl.clip_grads(grads, 1e9)                          # within it: no value changes
        assert all(torch.equal(g, (b.float() * scale).to(b.dtype)) for g, b in zip(grads, before))
        assert all(g._version > v for g, v in zip(grads, version))


@gpu
def test_missing_gradients_repeated_calls_and_workspaces():
    grads = tensors([50, 100000, 3], TYPES, 2)
    want = rl.grad_norm(grads)
    assert torch.equal(rl.grad_norm([None, grads[0], None, grads[1], grads[2], None]), want)
    assert all(torch.equal(rl.grad_norm(grads), want) for _ in range(5))
    twice = rl.grad_norm([grads[1], grads[1]])
    near(twice, norm_of([grads[1], grads[1]]), 1.01)
    sizes = (ctypes.c_int64 * 3)(50, 100000, 3)
    nbytes = rl.library().rlpl_grad_norm_workspace_bytes(sizes, 3)
    ws = torch.full((nbytes + 256,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(rl.grad_norm(grads, workspace=ws), want)
    with pytest.raises(rl.RlplError):
        rl.grad_norm(grads, workspace=ws[:100])


@gpu
def test_the_optimizer_takes_the_factor():
    """grad_norm's scale as adamw_step's grad_scale is the step with clipped gradients."""
    for dtype in (torch.float32, torch.bfloat16):
        params = tensors([1000, 33, 70001], [torch.float32], 1)
        other = [p.clone() for p in params]
        grads = tensors([1000, 33, 70001], [dtype], 2)
        a, b = rl.adamw_plan(params), rl.adamw_plan(other)
        for step in (1, 2):
            _, scale = rl.grad_norm(grads, max_norm=1.0)
            rl.adamw_step(a, grads, step=step, lr=1e-2, grad_scale=scale)
            wide = [g.float() * scale for g in grads]       # the optimizer's own first operation
            rl.adamw_step(b, wide, step=step, lr=1e-2)
            assert all(torch.equal(x, y) for x, y in zip(params, other))


@gpu
def test_another_stream_and_a_replayed_graph():
    grads = tensors(LISTS["two windows"] + [200000], TYPES, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = rl.grad_norm(grads, max_norm=1.0)
    with torch.cuda.stream(side):
        got = rl.grad_norm(grads, max_norm=1.0)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    saved = [g.clone() for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = rl.clip_grads(grads, 0.5)
    for i in range(1, 4):
        for g, s in zip(grads, saved):
            g.copy_(s * i)
        graph.replay()
        torch.cuda.synchronize()
        eager = [s * i for s in saved]
        assert torch.equal(rl.clip_grads(eager, 0.5), norm)
        assert all(torch.equal(x, y) for x, y in zip(grads, eager))


@gpu
def test_a_saved_gradient_that_was_scaled_is_noticed():
    x = torch.randn(10, device=DEV, requires_grad=True)
    g = torch.randn(10, device=DEV)
    loss = (x * g).sum()
    rl.scale_grads([g], torch.tensor(0.5, device=DEV))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@gpu
def test_past_32_bits_of_elements():
    n = 2 ** 31 + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[-5:] = 3.0
    g[2 ** 31 - 1] = 4.0
    near(rl.grad_norm([g]), math.sqrt(5 * 9 + 16), 1.01)
    rl.scale_grads([g], torch.tensor(0.5, device=DEV))
    assert (g[-5:] == 1.5).all() and g[2 ** 31 - 1] == 2.0 and g[-6] == 0


@gpu
def test_refusals_of_tensors():
    g, s = torch.zeros(8, device=DEV), torch.ones((), device=DEV)
    for bad, error in [([], ValueError), ([None], ValueError), ([g.cpu()], TypeError), ([g.int()], TypeError), ([3.0], TypeError),
                       ([g, torch.eye(3, device=DEV).to_sparse()], TypeError)]:
        with pytest.raises(error):
            rl.grad_norm(bad)
        with pytest.raises(error):
            rl.scale_grads(bad, s)
    with pytest.raises(ValueError):
        rl.grad_norm([g], norm_type=1.0)
    for bad in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(max_norm=1.0, eps=-1.0)):
        with pytest.raises(rl.RlplError):
            rl.grad_norm([g], **bad)
    with pytest.raises(TypeError):
        rl.grad_norm([g], grad_scale=s.double())
    with pytest.raises(TypeError):
        rl.scale_grads([g], torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        rl.scale_grads([g[::2]], s)
    with pytest.raises(ValueError):
        rl.scale_grads([g[:1].expand(4)], s)
    with pytest.raises(ValueError):
        rl.clip_grads([g], None)
    for twice in ([g, g], [g[:5], g[4:]], [g[6:], g[:3], g[2:4]], [g, torch.zeros(3, device=DEV), g[3:4]]):
        with pytest.raises(rl.RlplError):
            rl.scale_grads(twice, s)


def c_lists(sizes, dtypes=None, at=0x7F0000000000):
    n = len(sizes)
    pointers, place = [], at
    for s in sizes:
        pointers.append(place if s else None)
        place += max(0, s) * 4 + 16
    return (ctypes.c_void_p * n)(*pointers), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*(dtypes or [0] * n)), n


def test_refusals_of_the_c_entries():
    lib = rl.library()
    P = ctypes.c_void_p(0x7F0000000000)
    odd = ctypes.c_void_p(0x7F0000000002)

    def norm(lists=None, kind=0, gs=None, max_norm=1.0, eps=1e-6, out=P, scale=P, ws=P, wn=1 << 30):
        return lib.rlpl_grad_norm(*(lists or c_lists([5, 0, 9])), kind, gs, max_norm, eps, out, scale, ws, wn, None)

    def scale(lists=None, s=P):
        return lib.rlpl_grad_scale(*(lists or c_lists([5, 0, 9])), s, None)

    assert norm() == 7 and scale() == 7 or torch.cuda.is_available()
    for f in (norm, scale):
        assert f(c_lists([5, -1])) == 2 and f(c_lists([(1 << 40) + 1])) == 2 and f(c_lists([5], [3])) == 4
        p, s, d, n = c_lists([5, 6])
        assert f((None, s, d, n)) == 1 and f((p, None, d, n)) == 1 and f((p, s, None, n)) == 1 and f((p, s, d, 0)) == 2
        p[1] = None
        assert f((p, s, d, n)) == 1
        p[1] = 0x7F0000000002
        assert f((p, s, d, n)) == 3
    assert norm(kind=2) == 5 and norm(max_norm=-1.0) == 5 and norm(max_norm=math.inf) == 5 and norm(eps=math.nan) == 5
    assert norm(out=None) == 1 and norm(out=odd) == 3 and norm(scale=odd) == 3 and norm(gs=odd) == 3
    assert norm(ws=None) == 6 and norm(wn=8) == 6 and norm(ws=ctypes.c_void_p(0x7F0000000010)) == 3
    assert scale(s=None) == 1 and scale(s=odd) == 3
    p, s, d, n = c_lists([5, 6])
    p[1] = p[0]
    assert scale((p, s, d, n)) == 5
    assert scale(((ctypes.c_void_p * 2)(0x7F0000001000, 0x7F0000000000), (ctypes.c_int64 * 2)(4, 1025), d, 2)) == 5
    size = lambda sizes: lib.rlpl_grad_norm_workspace_bytes((ctypes.c_int64 * len(sizes))(*sizes), len(sizes))  # noqa: E731
    assert size([0]) == size([1]) == size([1] * 190) == 2048 * 8 and size([1] * 191) == 2 * 2048 * 8
    assert size([1 << 40] * 7) == 2048 * 8 and size([1 << 40] * 8) == 2 * 2048 * 8 and size([-1]) == 0
    assert lib.rlpl_grad_norm_workspace_bytes(None, 3) == 0
