"""The AdamW step: against numpy's float32 bit for bit (tests/adamw_reference.py), and against float64.

Every operation of the step is one correctly rounded float32 operation in a fixed order, on both sides, so
parameters, moments, 8-bit codes and scales are compared for equality.  Against float64 (eps = 2^-24, the most a
float32 operation is off): m is off by 4 eps (|b1 m| + |c1 g|) (two products, a sum, the coefficients' own rounding),
v by 6 eps v (all terms positive, c2 g g twice rounded), so sqrt(v) root + eps by 6 eps relative, the update by
lr / c * err(m) / denom + 12 eps |u|, and p by that and 3 eps |p|.
"""
import ctypes

import numpy as np
import pytest
import torch

import adamw_reference as ref
import rl_post_loss_amd as rl

DEV = "cuda:0"
E32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
gpu = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def tensors(sizes, seed, scale=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale * torch.exp(torch.randn(n, generator=g))).to(dtype) for n in sizes]


def on_device(ts):
    return [t.to(DEV) for t in ts]


def bits(t):
    t = t.detach().cpu()
    if t.dtype == F8:
        return t.view(torch.uint8).numpy()
    return t.view(torch.int16).numpy() if t.element_size() == 2 else t.view(torch.int32).numpy()


def same(name, got, want):
    got, want = bits(got), want if isinstance(want, np.ndarray) else bits(want)
    assert got.dtype == want.dtype and np.array_equal(got, want), \
        f"{name}: {(got != want).sum()} of {got.size} differ, first at {np.argmax(got != want)}"


def f32_bits(a):
    return np.asarray(a, dtype=np.float32).view(np.int32)


SIZES = [1, 2, 3, 5, 255, 256, 257, 1000, 4095, 4096, 4097, 12289, 0, 65536, 100003]
HYPER = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8)


def run_steps(sizes, bits_, pdt, gdt, cdt, steps=3, scale=None, seed=5, first=1, **over):
    hyper = {**HYPER, **over}
    p0 = tensors(sizes, 1, 0.1, DT[pdt])
    params = on_device(p0)
    copies = [torch.zeros_like(p, dtype=DT[cdt]) for p in params] if cdt else None
    decay = [0.1 * (i % 3) for i in range(len(sizes))]
    plan = rl.adamw_plan(params, state_dtype=F8 if bits_ == 8 else torch.float32, weight_decay=decay, copies=copies)
    p = [t.float().numpy().copy() for t in p0]
    m = [np.zeros(n, np.float32) for n in sizes]
    v = [np.zeros(n, np.float32) for n in sizes]
    mq, rq = ([np.zeros(n, np.uint8) for n in sizes] for _ in range(2))
    ms, rs = ([np.zeros((n + 255) // 256, np.float32) for n in sizes] for _ in range(2))
    sc = torch.tensor([scale], device=DEV) if scale is not None else None
    for t in range(first, first + steps):
        grads = tensors(sizes, 100 + t, 0.01, DT[gdt])
        rl.adamw_step(plan, on_device(grads), step=t, seed=seed, grad_scale=sc, **hyper)
        k = ref.coefficients(hyper["lr"], hyper["betas"], hyper["eps"], t)
        for i, g in enumerate(grads):
            g = g.float().numpy()
            if scale is not None:
                g = g * np.float32(scale)
            if bits_ == 8:
                m0, r0 = ref.decode(mq[i], ms[i]), ref.decode(rq[i], rs[i])
                p[i], mm, r, _ = ref.step(p[i], g, m0, r0 * r0, k, decay[i])
                w = ref.random_words(seed, t, i, g.size)
                mq[i], ms[i] = ref.encode(mm, w & np.uint64(0xFFFF), False)
                rq[i], rs[i] = ref.encode(r, w >> np.uint64(16), True)
            else:
                p[i], m[i], _, v[i] = ref.step(p[i], g, m[i], v[i], k, decay[i])
            if pdt != "fp32":
                p[i] = torch.from_numpy(p[i]).to(DT[pdt]).float().numpy()
        for i in range(len(sizes)):
            at = f"step {t}, tensor {i} of {sizes[i]}"
            if bits_ == 8:
                same(at + " exp_avg", plan.exp_avg[i], mq[i])
                same(at + " exp_avg_scale", plan.exp_avg_scale[i], f32_bits(ms[i]))
                same(at + " exp_avg_sq", plan.exp_avg_sq[i], rq[i])
                same(at + " exp_avg_sq_scale", plan.exp_avg_sq_scale[i], f32_bits(rs[i]))
            else:
                same(at + " exp_avg", plan.exp_avg[i], f32_bits(m[i]))
                same(at + " exp_avg_sq", plan.exp_avg_sq[i], f32_bits(v[i]))
            same(at + " param", params[i], torch.from_numpy(p[i]).to(DT[pdt]))
            if cdt:
                same(at + " copy", copies[i], torch.from_numpy(p[i]).to(DT[cdt]))
    return plan


@gpu
@pytest.mark.parametrize("gdt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pdt,cdt", [("fp32", None), ("fp32", "bf16"), ("fp32", "fp16"), ("bf16", None), ("fp16", None)])
@pytest.mark.parametrize("state", [32, 8])
def test_equal_to_numpy(state, pdt, cdt, gdt):
    run_steps(SIZES, state, pdt, gdt, cdt)


@gpu
@pytest.mark.parametrize("state", [32, 8])
def test_gradient_scale_late_steps_and_other_betas(state):
    run_steps([300, 5000], state, "fp32", "bf16", "bf16", scale=0.37, first=123456, seed=0xDEADBEEF)
    run_steps([300, 5000], state, "fp32", "fp32", None, betas=(0.0, 0.95), eps=1e-6, lr=0.0)


@gpu
@pytest.mark.parametrize("state", [32, 8])
def test_more_tensors_than_one_launch_takes(state):
    run_steps([7 + 31 * (i % 40) for i in range(1000)], state, "fp32", "bf16", "bf16", steps=1)


@gpu
@pytest.mark.parametrize("state", [32, 8])
def test_tensors_that_start_off_16_bytes(state):
    """Views into a flat buffer at odd offsets, for parameters, gradients and states, and their neighbours' bytes."""
    sizes = [257, 4100, 33]
    flat = torch.full((sum(sizes) + 8,), 3.0, device=DEV)
    gflat = torch.zeros(sum(sizes) + 8, dtype=torch.bfloat16, device=DEV)
    views, grads, at = [], [], 1
    for n, p, g in zip(sizes, tensors(sizes, 1, 0.1), tensors(sizes, 2, 0.01, torch.bfloat16)):
        views.append(flat[at:at + n])
        views[-1].copy_(p)
        grads.append(gflat[at:at + n])
        grads[-1].copy_(g)
        at += n + 1
    before = flat.clone()
    aligned = [v.clone() for v in views]
    kw = dict(state_dtype=F8 if state == 8 else torch.float32)
    a, b = rl.adamw_plan(views, **kw), rl.adamw_plan(aligned, **kw)
    for t in (1, 2):
        rl.adamw_step(a, grads, step=t, **HYPER)
        rl.adamw_step(b, [g.clone() for g in grads], step=t, **HYPER)
    for i in range(3):
        same("param", views[i], aligned[i])
        same("exp_avg", a.exp_avg[i], b.exp_avg[i])
        same("exp_avg_sq", a.exp_avg_sq[i], b.exp_avg_sq[i])
    gaps = [0, 258, 258 + 4101, 258 + 4101 + 34]
    assert torch.equal(flat[gaps], before[gaps])


@gpu
def test_against_float64():
    sizes = [10000]
    plan = rl.adamw_plan(on_device(tensors(sizes, 1, 0.1)), weight_decay=0.05)
    p, m, v = tensors(sizes, 1, 0.1)[0].double(), torch.zeros(10000).double(), torch.zeros(10000).double()
    tm = torch.zeros(10000).double()
    for t in range(1, 4):
        g = tensors(sizes, 50 + t, 0.01)[0]
        prev = [x[0].cpu().double() for x in (plan.params, plan.exp_avg, plan.exp_avg_sq)]
        rl.adamw_step(plan, [g.to(DEV)], step=t, **HYPER)
        p, m, v = prev                                  # one step at a time, from the state held
        g = g.double()
        tm = 4 * E32 * ((0.9 * m).abs() + (0.1 * g).abs())
        m = 0.9 * m + 0.1 * g
        v = 0.999 * v + 0.001 * g * g
        denom = (v / (1 - 0.999 ** t)).sqrt() + 1e-8
        u = 1e-2 / (1 - 0.9 ** t) * m / denom
        tp = 1e-2 / (1 - 0.9 ** t) * tm / denom + 12 * E32 * u.abs() + 3 * E32 * p.abs()
        want = p * (1 - 1e-2 * 0.05) - u
        assert ((plan.exp_avg[0].cpu().double() - m).abs() <= tm).all()
        assert ((plan.exp_avg_sq[0].cpu().double() - v).abs() <= 6 * E32 * v + 1e-45).all()
        assert ((plan.params[0].cpu().double() - want).abs() <= tp).all()


@gpu
@pytest.mark.parametrize("state", [32, 8])
def test_step_and_rate_on_the_device_and_in_a_graph(state):
    """Device scalars give what numbers give, and a captured step replayed with others is the eager step."""
    kw = dict(state_dtype=F8 if state == 8 else torch.float32)
    p = tensors([700, 5000], 1, 0.1)
    a, b = rl.adamw_plan(on_device(p), **kw), rl.adamw_plan(on_device(p), **kw)
    grads = on_device(tensors([700, 5000], 2, 0.01))
    step, lr = torch.ones(1, dtype=torch.int64, device=DEV), torch.tensor([1e-2], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rl.adamw_step(a, grads, step=step, lr=lr, seed=9)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rl.adamw_step(a, grads, step=step, lr=lr, seed=9)
    lrs = [1e-2] + [1e-2 * t for t in (2, 3, 4, 5)]
    for t in range(1, 6):
        if t > 1:
            step.fill_(t)
            lr.fill_(lrs[t - 1])
            for g, new in zip(grads, tensors([700, 5000], 2 + t, 0.01)):
                g.copy_(new)
            torch.cuda.synchronize()
            graph.replay()
        rl.adamw_step(b, [g.clone() for g in grads], step=t, lr=float(np.float32(lrs[t - 1])), seed=9)
        torch.cuda.synchronize()
        for i in range(2):
            same(f"step {t} param", a.params[i], b.params[i])
            same(f"step {t} exp_avg", a.exp_avg[i], b.exp_avg[i])
            same(f"step {t} exp_avg_sq", a.exp_avg_sq[i], b.exp_avg_sq[i])


@gpu
@pytest.mark.parametrize("state", [32, 8])
def test_bad_gradients_stay_in_their_element(state):
    kw = dict(state_dtype=F8 if state == 8 else torch.float32)
    p = tensors([600], 1, 0.1)
    a, b = rl.adamw_plan(on_device(p), **kw), rl.adamw_plan(on_device(p), **kw)
    g = tensors([600], 2, 0.01)[0]
    bad = g.clone()
    bad[3], bad[300] = float("nan"), float("inf")
    zeroed = g.clone()
    zeroed[[3, 300]] = 0.0
    rl.adamw_step(a, [bad.to(DEV)], step=1, **HYPER)
    rl.adamw_step(b, [zeroed.to(DEV)], step=1, **HYPER)
    keep = [i for i in range(600) if i not in (3, 300)]
    for x, y in ((a.params[0], b.params[0]), *zip(a.moments(0), b.moments(0))):
        assert torch.equal(x[keep], y[keep]) and not torch.isfinite(x[[3, 300]]).any()


@gpu
@pytest.mark.parametrize("state", [32, 8])
def test_no_gradient_leaves_a_tensor_and_an_empty_one_is_taken(state):
    kw = dict(state_dtype=F8 if state == 8 else torch.float32)
    params = on_device(tensors([50, 0, 300], 1, 0.1))
    before = [p.clone() for p in params]
    plan = rl.adamw_plan(params, **kw)
    g = on_device(tensors([50, 0, 300], 2, 0.01))
    rl.adamw_step(plan, [None, g[1], g[2]], step=1, **HYPER)
    assert torch.equal(params[0], before[0]) and not torch.equal(params[2], before[2])
    assert not bits(plan.exp_avg[0]).any()
    rl.adamw_step(plan, [None, None, None], step=2, **HYPER)
    rl.adamw_step(rl.adamw_plan([torch.zeros(0, device=DEV)]), [torch.zeros(0, device=DEV)], step=1, lr=0.1)


@gpu
def test_random_rounding_is_right_on_average():
    """One element's moment after a step, over 4096 seeds: the mean is within 5 standard errors of the value.  A
    rounding between neighbours d apart has a deviation of at most d / 2; e4m3 neighbours are at most 1/8 of the value
    apart."""
    n, seeds = 256, 4096
    g = tensors([n], 7, 0.01)[0].to(DEV)
    total_m, total_r = torch.zeros(n, device=DEV, dtype=torch.float64), torch.zeros(n, device=DEV, dtype=torch.float64)
    for s in range(seeds):
        plan = rl.adamw_plan([torch.zeros(n, device=DEV)], state_dtype=F8)
        rl.adamw_step(plan, [g], step=1, lr=0.0, seed=s)
        m, v = plan.moments(0)
        total_m += m.double()
        total_r += v.double().sqrt()
    want_m, want_r = 0.1 * g.double(), (0.001 * g.double() ** 2).sqrt()
    for total, want in ((total_m, want_m), (total_r, want_r)):
        big = want.abs() > want.abs().max() / 448 * 2.0 ** -6   # e4m3's normal range
        off = (total / seeds - want).abs()[big] / want.abs()[big]
        assert (off <= 5 * (1 / 16) / seeds ** 0.5).all()


@gpu
def test_moments_resumed_from_given_tensors_and_in_their_shape():
    p = tensors([35 * 20], 1, 0.1)[0].view(35, 20).to(DEV)
    a = rl.adamw_plan([p.clone()], state_dtype=F8, weight_decay=0.0)
    g = [tensors([700], 3 + t, 0.01)[0].view(35, 20).to(DEV) for t in range(3)]
    rl.adamw_step(a, [g[0]], step=1, **HYPER)
    assert a.exp_avg[0].shape == (35, 20) and a.moments(0)[0].shape == (35, 20)
    b = rl.adamw_plan([a.params[0].clone()], exp_avg=[a.exp_avg[0].clone()], exp_avg_sq=[a.exp_avg_sq[0].clone()],
                      exp_avg_scale=[a.exp_avg_scale[0].clone()], exp_avg_sq_scale=[a.exp_avg_sq_scale[0].clone()],
                      weight_decay=0.0)
    for t in (2, 3):
        rl.adamw_step(a, [g[t - 1]], step=t, **HYPER)
        rl.adamw_step(b, [g[t - 1].t().contiguous().t()], step=t, **HYPER)    # a gradient in another layout
    same("param", a.params[0], b.params[0])
    same("exp_avg", a.exp_avg[0], b.exp_avg[0])


@gpu
def test_a_graph_that_saved_an_old_value_says_so():
    p = torch.nn.Parameter(torch.ones(300, device=DEV))
    copy = torch.ones(300, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    plan = rl.adamw_plan([p], copies=[copy])
    losses = [(p * p).sum(), (copy * copy).sum()]
    rl.adamw_step(plan, [torch.ones(300, device=DEV)], step=1, **HYPER)
    for loss in losses:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    (p * p).sum().backward()
    assert torch.equal(p.grad, 2 * p.detach())
    loss = (p * p).sum()
    rl.adamw_step(plan, [None], step=2, **HYPER)         # nothing was written
    loss.backward()


# ------------------------------------------------------------------------------------------------------- refusals

A = 0x7F0000001000


def build(sizes=(8, 300), pdt=0, cdt=None, state=32, decay=(0.0, 0.1), plan=True, nbytes=None, **over):
    lib, n = rl.library(), len(sizes)
    cs = (ctypes.c_int64 * n)(*sizes)
    ptrs = lambda off, name: (ctypes.c_void_p * n)(*over.get(name, [A + off + 0x10000 * i for i in range(n)]))  # noqa: E731
    want = lib.rlpl_adamw_plan_bytes(cs, n)
    buf = np.zeros(max(want, 64) // 8 + 1, np.uint64)
    st = lib.rlpl_adamw_plan_build(
        buf.ctypes.data if plan else None, want if nbytes is None else nbytes, cs, n, ptrs(0, "p"), pdt,
        ptrs(0x100000, "c") if cdt is not None else None, cdt or 0, ptrs(0x200000, "m"), ptrs(0x300000, "v"),
        ptrs(0x400000, "ms") if state == 8 and "no_scale" not in over else None, ptrs(0x500000, "vs") if state == 8 else None,
        state, (ctypes.c_double * n)(*decay))
    return rl.STATUS[st], buf


def test_refusals_of_the_plan():
    for state in (32, 8):
        assert build(state=state)[0] == "RLPL_OK"
        assert build(state=state, cdt=2)[0] == "RLPL_OK"
    assert build(sizes=(0, 5), p=[None, A], m=[None, A + 0x1000], v=[None, A + 0x2000])[0] == "RLPL_OK"
    for want, over in [("RLPL_ERR_NULL", dict(plan=False)), ("RLPL_ERR_NULL", dict(p=[A, None])),
                       ("RLPL_ERR_NULL", dict(state=8, no_scale=True)), ("RLPL_ERR_NULL", dict(state=8, vs=[None, A])),
                       ("RLPL_ERR_SHAPE", dict(sizes=(-1, 5))), ("RLPL_ERR_SHAPE", dict(sizes=((1 << 40) + 1, 5))),
                       ("RLPL_ERR_DTYPE", dict(pdt=3)), ("RLPL_ERR_DTYPE", dict(state=16)),
                       ("RLPL_ERR_DTYPE", dict(cdt=0)), ("RLPL_ERR_DTYPE", dict(pdt=2, cdt=2)),
                       ("RLPL_ERR_ALIGN", dict(p=[A + 2, A + 0x1000])), ("RLPL_ERR_ALIGN", dict(m=[A + 2, A + 0x1000])),
                       ("RLPL_ERR_ALIGN", dict(state=8, ms=[A + 2, A + 0x1000])),
                       ("RLPL_ERR_WORKSPACE", dict(nbytes=100)), ("RLPL_ERR_PARAM", dict(decay=(0.0, -0.1))),
                       ("RLPL_ERR_PARAM", dict(decay=(float("nan"), 0.0)))]:
        assert build(**over)[0] == want, over
    assert rl.library().rlpl_adamw_plan_bytes(None, 3) == 0
    assert rl.library().rlpl_adamw_plan_bytes((ctypes.c_int64 * 1)(5), 0) == 0


def test_refusals_of_the_step():
    buf = build()[1]
    wrong = buf.copy()
    wrong[0] = 7

    def call(**over):
        a = dict(plan=buf.ctypes.data, dev=A, grads=(A, A + 64), gdt=2, lr=0.1, lr_at=None, b1=0.9, b2=0.99, eps=1e-8,
                 step=1, step_at=None, scale=None)
        a.update(over)
        g = (ctypes.c_void_p * 2)(*a["grads"]) if a["grads"] else None
        return rl.STATUS[rl.library().rlpl_adamw_step(a["plan"], a["dev"], g, a["gdt"], a["lr"], a["lr_at"], a["b1"],
                                                      a["b2"], a["eps"], a["step"], a["step_at"], a["scale"], 0, None)]

    for want, over in [("RLPL_ERR_NULL", dict(plan=None)), ("RLPL_ERR_NULL", dict(dev=None)),
                       ("RLPL_ERR_NULL", dict(grads=None)), ("RLPL_ERR_DTYPE", dict(gdt=3)),
                       ("RLPL_ERR_ALIGN", dict(grads=(A + 1, A))), ("RLPL_ERR_ALIGN", dict(dev=A + 4)),
                       ("RLPL_ERR_ALIGN", dict(scale=A + 2)), ("RLPL_ERR_ALIGN", dict(step_at=A + 4)),
                       ("RLPL_ERR_PARAM", dict(lr=-1.0)), ("RLPL_ERR_PARAM", dict(lr=float("inf"))),
                       ("RLPL_ERR_PARAM", dict(b1=1.0)), ("RLPL_ERR_PARAM", dict(b2=-0.1)),
                       ("RLPL_ERR_PARAM", dict(b2=float("nan"))), ("RLPL_ERR_PARAM", dict(eps=-1e-8)),
                       ("RLPL_ERR_PARAM", dict(step=0)), ("RLPL_ERR_PARAM", dict(plan=wrong.ctypes.data))]:
        assert call(**over) == want, over
    if not torch.cuda.is_available():
        assert call() == "RLPL_ERR_DEVICE" and call(grads=(None, A)) == "RLPL_ERR_DEVICE"


def test_refusals_of_the_binding_on_the_host():
    with pytest.raises(ValueError):
        rl.adamw_plan([])
    with pytest.raises(TypeError):
        rl.adamw_plan([torch.zeros(4)])


@gpu
def test_refusals_of_the_binding():
    z = lambda n=8, dt=torch.float32: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
    p = z()
    for want, args, kw in [(TypeError, [p, z(8, torch.bfloat16)], {}), (TypeError, [z(8, torch.float64)], {}),
                           (ValueError, [z(16)[::2]], {}), (ValueError, [p, p], {}), (ValueError, [p, p[4:]], {}),
                           (ValueError, [p], dict(copies=[])), (TypeError, [p], dict(copies=[z()])),
                           (ValueError, [p], dict(copies=[z(9, torch.bfloat16)])),
                           (ValueError, [z(8, torch.bfloat16)], dict(copies=[z(8, torch.bfloat16)])),
                           (TypeError, [p], dict(state_dtype=torch.float16)), (ValueError, [p], dict(exp_avg=[z()])),
                           (ValueError, [p], dict(exp_avg=[z()], exp_avg_sq=[z()], exp_avg_scale=[z(1)])),
                           (ValueError, [p], dict(weight_decay=[0.1, 0.1])),
                           (ValueError, [p], dict(exp_avg=[z()], exp_avg_sq=[p]))]:
        with pytest.raises(want):
            rl.adamw_plan(args, **kw)
    with pytest.raises(rl.RlplError, match="PARAM"):
        rl.adamw_plan([p], weight_decay=-1.0)
    plan = rl.adamw_plan([p])
    for want, grads, kw in [(ValueError, [], {}), (ValueError, [z(9)], {}), (ValueError, [z(8).view(2, 4)], {}),
                            (ValueError, [torch.zeros(8)], {}), (TypeError, [z(8, torch.float64)], {}),
                            (TypeError, [z()], dict(step=torch.ones(1, device=DEV))),
                            (TypeError, [z()], dict(grad_scale=torch.ones(2, device=DEV)))]:
        with pytest.raises(want):
            rl.adamw_step(plan, grads, **{**dict(step=1, lr=0.1), **kw})
    with pytest.raises(rl.RlplError, match="PARAM"):
        rl.adamw_step(plan, [z()], step=0, lr=0.1)
