"""Measured cases of the operators around the losses of a training step.

The framework's losses start from the last hidden states and an output projection and end in gradients.  Three
operators surround them: the layer norm that makes those hidden states, the softmax cross entropy of the projection
over a large vocabulary (supervised tokens, next to the selective log-probabilities), and the AdamW step that uses
the gradients.  Each has a plain form here, in elementary torch operations, and the framework's call.

    ce     loss = sum_i (lse_i - z_i[y_i] + z_loss * lse_i^2) / max(N, 1) over the N rows whose target is not ignored,
           z_i = hidden_i . weight^T + bias, with the gradients of hidden, weight and bias (or the loss alone)
    ln     y = (x - mean) * rstd * weight + bias per row, and its backward pass with the weight's and bias's gradients
    adamw  one step over a list of tensors, states in float32 or in 8 bits (e4m3, one scale for 256 values, the
           second moment by its square root, rounded at random by numbers made from a seed)
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORE = -100
BLOCK = 256             # values of an 8-bit state that share one scale
TOP = 448.0             # the largest e4m3 value
INV_TOP = float(np.float32(1.0) / np.float32(448.0))
TINY = 2.0 ** -118      # a block whose largest value is below this is held as zeros
M32 = 0xFFFFFFFF


def listed():
    return [
        # a short ragged batch (a unit test's or a draft model's size): latency of the whole call
        {"name": "ce_bf16_200x512x2051", "op": "ce", "n": 200, "H": 512, "V": 2051, "dtype": "bf16", "bias": True,
         "grad": True, "ignored": 0.25, "z_loss": 0.0},
        # a few supervised tokens against a full projection: bound by the weight's traffic
        {"name": "ce_bf16_16x4096x128256", "op": "ce", "n": 16, "H": 4096, "V": 128256, "dtype": "bf16", "bias": False,
         "grad": True, "ignored": 0.0, "z_loss": 0.0},
        # one group of tokens at the size the log-probabilities are timed at
        {"name": "ce_bf16_1024x4096x128256", "op": "ce", "n": 1024, "H": 4096, "V": 128256, "dtype": "bf16",
         "bias": True, "grad": True, "ignored": 0.0, "z_loss": 0.0},
        # packed sequences with their prompts ignored, a vocabulary that ends inside a tile, the z penalty
        {"name": "ce_fp16_6001x2048x50021", "op": "ce", "n": 6001, "H": 2048, "V": 50021, "dtype": "fp16",
         "bias": False, "grad": True, "ignored": 0.5, "z_loss": 1e-4},
        # evaluation: the loss alone
        {"name": "ce_loss_bf16_2048x4096x128256", "op": "ce", "n": 2048, "H": 4096, "V": 128256, "dtype": "bf16",
         "bias": False, "grad": False, "ignored": 0.0, "z_loss": 0.0},
        # one decoded token's norm
        {"name": "ln_fwd_bf16_1x4096", "op": "ln", "n": 1, "H": 4096, "dtype": "bf16", "bias": True, "grad": False},
        # a long packed batch's norm
        {"name": "ln_fwd_bf16_65536x4096", "op": "ln", "n": 65536, "H": 4096, "dtype": "bf16", "bias": True,
         "grad": False},
        # odd rows and columns in float32, no bias
        {"name": "ln_bwd_fp32_3001x1111", "op": "ln", "n": 3001, "H": 1111, "dtype": "fp32", "bias": False,
         "grad": True},
        # a training batch's backward pass
        {"name": "ln_bwd_bf16_32768x4096", "op": "ln", "n": 32768, "H": 4096, "dtype": "bf16", "bias": True,
         "grad": True},
        # a norm's and a bias's few small tensors: latency
        {"name": "adamw_fp32_6_small", "op": "adamw", "count": 6, "total": 24000, "state": "fp32", "grad_dtype": "fp32",
         "copy": "none", "step": 3},
        # a model's worth of tensors of all sizes, 16-bit gradients, float32 parameters with their 16-bit copies
        {"name": "adamw_fp32_300_mixed", "op": "adamw", "count": 300, "total": 150000000, "state": "fp32",
         "grad_dtype": "bf16", "copy": "bf16", "step": 1000},
        # one output projection with its moments in 8 bits
        {"name": "adamw_8bit_1_projection", "op": "adamw", "count": 1, "total": 128256 * 4096, "state": "8bit",
         "grad_dtype": "bf16", "copy": "bf16", "step": 100},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "ln", "adamw"])
    if op == "ce":
        grad = rng.random() < 0.75
        while True:
            n, H, V = _log_int(rng, 1, 8192), 8 * _log_int(rng, 2, 512), _log_int(rng, 8, 131072)
            if n * H * V <= 4.0e11:
                break
        return {"op": "ce", "n": n, "H": H, "V": V, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
                "bias": rng.random() < 0.5, "grad": grad, "ignored": rng.choice([0.0, 0.0, 0.25, 0.75]),
                "z_loss": rng.choice([0.0, 0.0, 1e-4, 1e-2])}
    if op == "ln":
        while True:
            n, H = _log_int(rng, 1, 65536), _log_int(rng, 2, 16384)
            if n * H <= 65536 * 2048:
                break
        if rng.random() < 0.5:
            H = max(8, H // 8 * 8)
        return {"op": "ln", "n": n, "H": H, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "bias": rng.random() < 0.7, "grad": rng.random() < 0.6}
    count = _log_int(rng, 1, 400)
    return {"op": "adamw", "count": count, "total": max(count, _log_int(rng, 100, 200000000)),
            "state": rng.choice(["fp32", "8bit"]), "grad_dtype": rng.choice(["bf16", "fp16", "fp32"]),
            "copy": rng.choice(["none", "bf16", "fp16"]), "step": _log_int(rng, 1, 100000)}


# ------------------------------------------------------------------------------------------------------- inputs

def _ignored_rows(n, share):
    """Rows whose target is ignored: the first `share` of every run of 128 rows, as prompts in packed sequences are
    (runs counted from the last row, which always counts)."""
    return [i for i in range(n) if (n - 1 - i) % 128 >= 128 * (1.0 - share)]


def _sizes(case):
    """Element counts of a list of `count` tensors that add up to about `total`: mostly small vectors of odd and even
    lengths, and a few large matrices, as the parameters of a model are."""
    count, total = case["count"], case["total"]
    if count == 1:
        return [total]
    r = np.random.RandomState(count * 7919 + total % 104729)
    w = np.exp(r.uniform(math.log(1.0), math.log(3e4), count))
    s = np.maximum(1, (w / w.sum() * total).astype(np.int64))
    s[r.rand(count) < 0.5] |= 1
    return [int(v) for v in s]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    if case["op"] == "ce":
        n, H, V, dt = case["n"], case["H"], case["V"], DTYPES[case["dtype"]]
        targets = torch.randint(0, V, (n,), device="cuda", generator=g)
        dropped = _ignored_rows(n, case["ignored"])
        if dropped:
            targets[torch.tensor(dropped, device="cuda")] = IGNORE
        return {"case": case, "hidden": randn(n, H, dtype=dt), "weight": randn(V, H, scale=2.0 / math.sqrt(H), dtype=dt),
                "bias": randn(V, scale=0.5, dtype=dt) if case["bias"] else None, "targets": targets}
    if case["op"] == "ln":
        n, H, dt = case["n"], case["H"], DTYPES[case["dtype"]]
        x = (randn(n, H, scale=1.5) + randn(n, 1)).to(dt)
        s = {"case": case, "x": x, "weight": (randn(H, scale=0.2) + 1.0).to(dt),
             "bias": randn(H, scale=0.2, dtype=dt) if case["bias"] else None}
        if case["grad"]:  # what the forward pass keeps
            xd = x.double()
            mean = xd.mean(dim=1)
            var = (xd - mean[:, None]).square().mean(dim=1)
            s |= {"grad_y": randn(n, H, dtype=dt), "mean": mean.float(), "rstd": (var + 1e-5).rsqrt().float()}
        return s
    sizes, eight = _sizes(case), case["state"] == "8bit"
    p, gr, m, v, sm, sv, cp = [], [], [], [], [], [], []
    for k in sizes:
        p.append(randn(k, scale=0.02))
        spread = torch.exp(randn(k, scale=1.0))          # coordinates of different gradient sizes
        gr.append((randn(k, scale=1e-3) * spread).to(DTYPES[case["grad_dtype"]]))
        first = 1e-3 * randn(k, scale=0.3) * spread
        second = (1e-3 * spread * (0.5 + torch.rand(k, device="cuda", generator=g))).square()
        if eight:
            q, s = _to_8bit(first, None, False)
            m.append(q), sm.append(s)
            q, s = _to_8bit(second.sqrt(), None, True)
            v.append(q), sv.append(s)
        else:
            m.append(first), v.append(second)
        if case["copy"] != "none":
            cp.append(p[-1].to(DTYPES[case["copy"]]))
        del spread, first, second
    decay = [0.01 if k > 1000 else 0.0 for k in sizes]
    s = {"case": case, "params": p, "grads": gr, "m": m, "v": v, "sm": sm, "sv": sv, "copies": cp, "decay": decay,
         "seed": int(seed) & M32}
    if own:
        import rl_post_loss_amd as rl
        s["plan"] = rl.adamw_plan(p, exp_avg=m, exp_avg_sq=v, exp_avg_scale=sm or None, exp_avg_sq_scale=sv or None,
                                  copies=cp or None, weight_decay=decay)
    return s


# ------------------------------------------------------------------------------------------------------- plain forms

LR, BETA1, BETA2, EPS = 1e-3, 0.9, 0.999, 1e-8


def _plain_ce(s):
    c, y = s["case"], s["targets"]
    h, w = s["hidden"].float(), s["weight"].float()
    z = h @ w.t()
    if s["bias"] is not None:
        z += s["bias"].float()
    valid = y != IGNORE
    at = torch.where(valid, y, 0)[:, None]
    inv = 1.0 / valid.sum().clamp(min=1).float()
    top = z.amax(dim=1, keepdim=True)
    target = z.gather(1, at)[:, 0]
    p = z.sub_(top).exp_()
    total = p.sum(dim=1)
    lse = top[:, 0] + total.log()
    rows = lse - target + c["z_loss"] * lse * lse
    loss = torch.where(valid, rows, 0.0).sum() * inv
    if not c["grad"]:
        return {"loss": loss}
    scale = torch.where(valid, inv, 0.0)
    dz = p.mul_((scale * (1.0 + 2.0 * c["z_loss"] * lse) / total)[:, None])
    dz.scatter_add_(1, at, -scale[:, None])
    out = {"loss": loss, "grad_hidden": (dz @ w).to(s["hidden"].dtype), "grad_weight": (dz.t() @ h).to(s["weight"].dtype)}
    if s["bias"] is not None:
        out["grad_bias"] = dz.sum(dim=0).to(s["bias"].dtype)
    return out


def _plain_ln(s):
    x, w = s["x"].float(), s["weight"].float()
    if not s["case"]["grad"]:
        mean = x.mean(dim=1)
        d = x - mean[:, None]
        rstd = (d.square().mean(dim=1) + 1e-5).rsqrt()
        y = d * rstd[:, None] * w
        if s["bias"] is not None:
            y += s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    dy = s["grad_y"].float()
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gy = dy * w
    dx = (gy - gy.mean(dim=1, keepdim=True) - n * (gy * n).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
    out = {"grad_x": dx.to(s["x"].dtype), "grad_weight": (dy * n).sum(dim=0).to(s["weight"].dtype)}
    if s["bias"] is not None:
        out["grad_bias"] = dy.sum(dim=0).to(s["bias"].dtype)
    return out


def _mix(x):
    """The 32-bit finalizer of MurmurHash3 (A. Appleby) on int64 tensors or numbers that hold 32-bit values."""
    x = x ^ (x >> 16)
    x = (x * 0x85EBCA6B) & M32
    x = x ^ (x >> 13)
    x = (x * 0xC2B2AE35) & M32
    return x ^ (x >> 16)


def _key(seed, step, tensor):
    return _mix(_mix(_mix(seed & M32) ^ (step & M32)) ^ tensor)


def _to_8bit(x, u, root):
    """x in blocks of 256 as e4m3 values and one float32 scale a block.  u: numbers in [0, 1) that decide each
    rounding (up where the part below the last place plus u reaches one), or None for one half throughout."""
    k = x.numel()
    blocks = (k + BLOCK - 1) // BLOCK
    a = torch.nn.functional.pad(x.abs(), (0, blocks * BLOCK - k)).view(blocks, BLOCK)
    finite = torch.isfinite(a)
    top = torch.where(finite, a, 0.0).amax(dim=1)
    live = top >= TINY
    scale = torch.where(live, top * INV_TOP, 0.0)
    inv = torch.where(live, torch.full_like(top, TOP) / top, 0.0)
    q = (a * inv[:, None]).view(-1)[:k]
    e = ((q.view(torch.int32) >> 23) - 127).clamp_(min=-6)          # the binade, e4m3's smallest normal one at least
    ulp = ((e + 124) << 23).view(torch.float32)                     # 2^(e - 3)
    per = ((130 - e) << 23).view(torch.float32)                     # 2^(3 - e)
    q = ((q * per + (0.5 if u is None else u)).floor() * ulp).clamp_(max=TOP)
    if root:
        q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)           # a second moment above zero stays above zero
    q = torch.where(torch.isfinite(x), torch.where(x < 0, -q, q), torch.full_like(q, float("nan")))
    return q.to(torch.float8_e4m3fn), scale


def _plain_adamw(s):
    c = s["case"]
    t = c["step"]
    step_size = float(np.float32(LR / (1.0 - BETA1 ** t)))
    root = float(np.float32(1.0 / math.sqrt(1.0 - BETA2 ** t)))
    params, grads = s["params"], [g.float() for g in s["grads"]]
    if c["state"] == "fp32":
        m, v = s["m"], s["v"]
        torch._foreach_mul_(m, BETA1)
        torch._foreach_add_(m, torch._foreach_mul(grads, float(np.float32(1.0 - BETA1))))
        torch._foreach_mul_(v, BETA2)
        torch._foreach_add_(v, torch._foreach_mul(torch._foreach_mul(grads, float(np.float32(1.0 - BETA2))), grads))
        denom = torch._foreach_sqrt(v)
        new_m = m
    else:
        pairs = [_plain_moments_8bit(s, i, grads[i], t) for i in range(len(params))]
        new_m, denom = [a for a, _ in pairs], [b for _, b in pairs]
    torch._foreach_mul_(denom, root)
    torch._foreach_add_(denom, EPS)
    update = torch._foreach_div(new_m, denom)
    torch._foreach_mul_(update, step_size)
    torch._foreach_mul_(params, [float(np.float32(1.0 - LR * d)) for d in s["decay"]])
    torch._foreach_sub_(params, update)
    if s["copies"]:
        torch._foreach_copy_(s["copies"], params)
    return _adamw_outputs(s)


def _plain_moments_8bit(s, i, g, t):
    """The new first moment and the second one's root of tensor i in float32, and its state updated in 8 bits."""
    k = g.numel()
    at = torch.arange(k, device=g.device)
    key = _key(s["seed"], t, i)
    word = _mix((at & M32) ^ _mix((key + (at >> 32)) & M32))
    per_block = lambda q, scale: q.float() * scale.repeat_interleave(BLOCK)[:k]  # noqa: E731
    m = per_block(s["m"][i], s["sm"][i]) * BETA1 + g * float(np.float32(1.0 - BETA1))
    r = per_block(s["v"][i], s["sv"][i])
    r = (r * r * BETA2 + g * float(np.float32(1.0 - BETA2)) * g).sqrt()
    for x, u, name, scale, root in ((m, word & 0xFFFF, "m", "sm", False), (r, word >> 16, "v", "sv", True)):
        q, sc = _to_8bit(x, u.float() * 2.0 ** -16, root)
        s[name][i].copy_(q)
        s[scale][i].copy_(sc)
    return m, r


def _whole(tensors):
    """All tensors of a list as one (64 outputs at most are wanted of a pass); the list's own tensor where it is one."""
    return tensors[0] if len(tensors) == 1 else torch.cat([t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in tensors]).view(tensors[0].dtype)


def _adamw_outputs(s):
    out = {"params": _whole(s["params"]), "exp_avg": _whole(s["m"]), "exp_avg_sq": _whole(s["v"])}
    if s["sm"]:
        out |= {"exp_avg_scale": _whole(s["sm"]), "exp_avg_sq_scale": _whole(s["sv"])}
    if s["copies"]:
        out["copies"] = _whole(s["copies"])
    return out


# ------------------------------------------------------------------------------------------------------- the calls

def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return {"ce": _plain_ce, "ln": _plain_ln, "adamw": _plain_adamw}[c["op"]](s)


def _own(s):
    import rl_post_loss_amd as rl
    c = s["case"]
    if c["op"] == "ce":
        if not c["grad"]:
            return {"loss": rl.linear_cross_entropy_fwd(s["hidden"], s["weight"], s["bias"], s["targets"],
                                                        z_loss=c["z_loss"])}
        loss, dh, dw, db = rl.linear_cross_entropy(s["hidden"], s["weight"], s["bias"], s["targets"],
                                                   z_loss=c["z_loss"])
        out = {"loss": loss, "grad_hidden": dh, "grad_weight": dw}
        return out if db is None else out | {"grad_bias": db}
    if c["op"] == "ln":
        if not c["grad"]:
            y, mean, rstd = rl.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=1e-5)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = rl.layer_norm_bwd(s["grad_y"], s["x"], s["weight"], s["mean"], s["rstd"],
                                       need_bias=s["bias"] is not None)
        out = {"grad_x": dx, "grad_weight": dw}
        return out if db is None else out | {"grad_bias": db}
    rl.adamw_step(s["plan"], s["grads"], step=c["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS, seed=s["seed"])
    return _adamw_outputs(s)


# ------------------------------------------------------------------------------------------------------- the work

def work(case):
    """Bytes: inputs read once, outputs written once.  Flops of ce: the logits, and two products for the gradients,
    over the rows that count; the rest by the terms of the formulas."""
    if case["op"] == "ce":
        n, H, V = case["n"] - len(_ignored_rows(case["n"], case["ignored"])), case["H"], case["V"]
        b = 2 * (n * H + V * H + (V if case["bias"] else 0)) + 8 * case["n"] + 4
        if case["grad"]:
            b += 2 * (case["n"] * H + V * H + (V if case["bias"] else 0))
        return {"bytes": b, "flops": (6 if case["grad"] else 2) * n * H * V}
    if case["op"] == "ln":
        n, H, e = case["n"], case["H"], 4 if case["dtype"] == "fp32" else 2
        vectors = (2 if case["bias"] else 1) * H * e
        if case["grad"]:
            return {"bytes": 3 * n * H * e + 8 * n + H * e + vectors, "flops": 14 * n * H}
        return {"bytes": 2 * n * H * e + 8 * n + vectors, "flops": 8 * n * H}
    sizes = _sizes(case)
    total = sum(sizes)
    b = total * (8 + (4 if case["grad_dtype"] == "fp32" else 2) + (0 if case["copy"] == "none" else 2))
    b += total * 16 if case["state"] == "fp32" else total * 4 + 16 * sum((k + BLOCK - 1) // BLOCK for k in sizes)
    return {"bytes": b, "flops": (16 if case["state"] == "fp32" else 50) * total}


# ------------------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ce":
        return _exact_ce(s)
    if case["op"] == "ln":
        return _exact_ln(s)
    return _exact_adamw(s)


def _exact_ce(s):
    """In groups of the rows that count, so that the logits in 64 bits fit beside the inputs."""
    c, y = s["case"], s["targets"]
    w = s["weight"].double()
    b = s["bias"].double() if s["bias"] is not None else None
    kept = torch.nonzero(y != IGNORE)[:, 0]
    count = max(1, kept.numel())
    loss = torch.zeros((), dtype=torch.float64, device=y.device)
    dh = torch.zeros(s["hidden"].shape, dtype=torch.float64, device=y.device)
    dw, db = torch.zeros_like(w), torch.zeros(w.shape[0], dtype=torch.float64, device=y.device)
    for rows in kept.split(1024):
        h = s["hidden"][rows].double()
        z = torch.matmul(h, w.t())
        if b is not None:
            z = z + b
        lse = torch.logsumexp(z, dim=1)
        hit = torch.zeros_like(z)
        hit[torch.arange(len(rows), device=y.device), y[rows]] = 1.0
        loss += (lse - (z * hit).sum(dim=1) + c["z_loss"] * lse ** 2).sum() / count
        if c["grad"]:
            d = ((1.0 + 2.0 * c["z_loss"] * lse)[:, None] * torch.exp(z - lse[:, None]) - hit) / count
            dh[rows] = torch.matmul(d, w)
            dw += torch.matmul(d.t(), h)
            db += d.sum(dim=0)
    out = {"loss": loss}
    if c["grad"]:
        out |= {"grad_hidden": dh, "grad_weight": dw}
        if b is not None:
            out["grad_bias"] = db
    return out


def _exact_ln(s):
    x, w = s["x"].double(), s["weight"].double()
    H = x.shape[1]
    if not s["case"]["grad"]:
        mean = x.sum(dim=1) / H
        var = ((x - mean[:, None]) ** 2).sum(dim=1) / H
        rstd = 1.0 / torch.sqrt(var + 1e-5)
        y = (x - mean[:, None]) * rstd[:, None] * w
        return {"y": y if s["bias"] is None else y + s["bias"].double(), "mean": mean, "rstd": rstd}
    mean, rstd, dy = s["mean"].double()[:, None], s["rstd"].double()[:, None], s["grad_y"].double()
    hat = (x - mean) * rstd
    d = dy * w
    # d/dx of sum(dy * y): the row's own term less the two that go through its mean and its variance
    dx = rstd * d - rstd / H * d.sum(dim=1, keepdim=True) - rstd / H * hat * (d * hat).sum(dim=1, keepdim=True)
    out = {"grad_x": dx, "grad_weight": torch.einsum("nh,nh->h", dy, hat)}
    if s["bias"] is not None:
        out["grad_bias"] = dy.sum(dim=0)
    return out


def _exact_adamw(s):
    """Parameters and moments from the formulas; an 8-bit state, which is a random rounding, has no value of its own."""
    c, eight = s["case"], s["case"]["state"] == "8bit"
    new = {"params": [], "exp_avg": [], "exp_avg_sq": []}
    for p, g, m, v, i in zip(s["params"], s["grads"], s["m"], s["v"], range(len(s["params"]))):
        g, k = g.double(), g.numel()
        if eight:
            at = torch.div(torch.arange(k, device=g.device), BLOCK, rounding_mode="floor")
            m = m.double() * s["sm"][i].double()[at]
            v = (v.double() * s["sv"][i].double()[at]) ** 2
        m = 0.9 * m.double() + (1.0 - 0.9) * g
        v = 0.999 * v.double() + (1.0 - 0.999) * g ** 2
        mhat, vhat = m / (1.0 - 0.9 ** c["step"]), v / (1.0 - 0.999 ** c["step"])
        new["params"].append(p.double() - LR * s["decay"][i] * p.double() - LR * mhat / (torch.sqrt(vhat) + EPS))
        new["exp_avg"].append(m)
        new["exp_avg_sq"].append(v)
        del g, m, v, mhat, vhat
    one = lambda t: t[0] if len(t) == 1 else torch.cat(t)  # noqa: E731
    out = {"params": one(new["params"]), "exp_avg": None if eight else one(new["exp_avg"]),
           "exp_avg_sq": None if eight else one(new["exp_avg_sq"])}
    if s["copies"]:
        out["copies"] = out["params"]
    return out
