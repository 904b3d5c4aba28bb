"""Measured cases of the operators that score tokens and of those around a training step's gradients.

A scoring pass goes from the last residual stream through a norm and an output projection to log-probabilities; a
training step ends in gradients that are clipped before the optimizer takes them.  Four operators, each with a plain
form here, in elementary torch operations, and the framework's call.

    logprobs  per row of logits z, at temperature T: logp = z[y]/T - lse, lse = log sum exp(z/T), the entropy
              H = lse - sum p z/T, and the k most likely tokens; or the gradient of g logp + h H with respect to z
    rms       h = x + residual, y = h / sqrt(avg(h^2) + eps) * weight, y in its type or in 8 bits (e4m3, a scale for
              every 128 columns); or the backward pass with the weight's gradient
    fp8       out = (x_q x_scale) . (w_q w_scale)^T of e4m3 operands, a scale for 128 columns of a row of x and for
              128 x 128 of w
    norm      the norm over a list of gradients and the factor that clips it; or the clipping itself, in place
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
GROUP = 128             # columns (and rows, of a projection) that share a scale
TOP = 448.0             # the largest e4m3 value
INV_TOP = float(np.float32(1.0) / np.float32(448.0))
TINY = 2.0 ** -118      # a group whose largest value is below this is held as zeros
EPS = 1e-6              # of the norm of rows
MAX_NORM, CLIP_EPS = 1.0, 1e-3   # clipping: gradients that were clipped before are over it again by CLIP_EPS


def listed():
    return [
        # eight sequences' next tokens while sampling, some of the vocabulary banned: latency of few long rows
        {"name": "logprobs_bf16_8x128256_top20", "op": "logprobs", "seqs": 1, "n": 8, "V": 128256, "dtype": "bf16",
         "grad": False, "top_k": 20, "T": 0.7, "masked": 0.0, "shifted": False, "banned": True},
        # scoring four packed sequences, their prompts masked, logits shifted by one against the tokens
        {"name": "logprobs_bf16_4x1024x128256", "op": "logprobs", "seqs": 4, "n": 1024, "V": 128256, "dtype": "bf16",
         "grad": False, "top_k": 5, "T": 1.0, "masked": 0.25, "shifted": True, "banned": False},
        # a policy step's gradient with an entropy bonus; rows of odd length
        {"name": "logprobs_bwd_fp16_3001x50021", "op": "logprobs", "seqs": 1, "n": 3001, "V": 50021, "dtype": "fp16",
         "grad": True, "top_k": 0, "T": 1.0, "masked": 0.25, "shifted": False, "banned": False},
        # one decoded token's norm on its way into an 8-bit projection
        {"name": "rms_fp8_bf16_1x4096", "op": "rms", "n": 1, "H": 4096, "dtype": "bf16", "grad": False, "fp8": True,
         "residual": "same"},
        # a long packed batch's norm
        {"name": "rms_fp8_bf16_32768x4096", "op": "rms", "n": 32768, "H": 4096, "dtype": "bf16", "grad": False,
         "fp8": True, "residual": "same"},
        # a training batch's backward pass, the stream's gradient joined
        {"name": "rms_bwd_bf16_16384x4096", "op": "rms", "n": 16384, "H": 4096, "dtype": "bf16", "grad": True,
         "fp8": False, "residual": "same"},
        # one token's logits: bound by the projection's bytes
        {"name": "fp8_1x4096x128256", "op": "fp8", "n": 1, "H": 4096, "V": 128256, "dtype": "bf16", "bias": False},
        # a ragged batch against a small odd projection
        {"name": "fp8_333x2048x5003", "op": "fp8", "n": 333, "H": 2048, "V": 5003, "dtype": "bf16", "bias": True},
        # a scored batch's logits
        {"name": "fp8_2048x4096x128256", "op": "fp8", "n": 2048, "H": 4096, "V": 128256, "dtype": "bf16", "bias": False},
        # a norm's and a bias's few small tensors: latency
        {"name": "norm_fp32_6_small", "op": "norm", "count": 6, "total": 24000, "dtype": "fp32", "inf": False,
         "clip": False},
        # a model's worth of gradients of all sizes; the factor goes to the optimizer
        {"name": "norm_bf16_300_mixed", "op": "norm", "count": 300, "total": 150000000, "dtype": "bf16", "inf": False,
         "clip": False},
        # gradients packed in one buffer, clipped in place
        {"name": "clip_fp32_300_mixed", "op": "norm", "count": 300, "total": 150000000, "dtype": "fp32", "inf": False,
         "clip": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "rms", "fp8", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "logprobs":
        grad = rng.random() < 0.4
        while True:
            seqs, n, V = rng.choice([1, 1, 2, 5]), _log_int(rng, 1, 4096), _log_int(rng, 64, 131072)
            if seqs * n * V <= (1.5e8 if grad or dtype == "fp32" else 5.2e8):
                break
        return {"op": "logprobs", "seqs": seqs, "n": n, "V": V, "dtype": dtype, "grad": grad,
                "top_k": 0 if grad else rng.choice([0, 1, 5, 20, 32]), "T": rng.choice([1.0, 1.0, 0.7, 1.3]),
                "masked": rng.choice([0.0, 0.25, 0.75]), "shifted": rng.random() < 0.5,
                "banned": not grad and rng.random() < 0.3}
    if op == "rms":
        grad, limit = rng.random() < 0.4, 16384 * 4096 if dtype == "fp32" else 32768 * 4096
        while True:
            n, H = _log_int(rng, 1, 65536), _log_int(rng, 2, 16384)
            if n * H <= (limit // 2 if grad else limit):
                break
        if rng.random() < 0.5:
            H = max(8, H // 8 * 8)
        return {"op": "rms", "n": n, "H": H, "dtype": dtype, "grad": grad, "fp8": not grad and rng.random() < 0.6,
                "residual": rng.choice(["none", "same", "fp32"])}
    if op == "fp8":
        while True:
            n, H, V = _log_int(rng, 1, 4096), 16 * _log_int(rng, 4, 512), _log_int(rng, 16, 131072)
            if n * H * V <= 1.0e12 and V * H <= 128256 * 4096:
                break
        return {"op": "fp8", "n": n, "H": H, "V": V, "dtype": dtype, "bias": rng.random() < 0.5}
    count, clip = _log_int(rng, 1, 400), rng.random() < 0.4
    return {"op": "norm", "count": count, "total": max(count, _log_int(rng, 100, 150000000)), "dtype": dtype,
            "inf": rng.random() < 0.25, "clip": clip}


# ------------------------------------------------------------------------------------------------------- inputs

def _masked_rows(n, share):
    """Rows that do not count: the first `share` of every run of 128 rows, as prompts in packed sequences are (runs
    counted from the last row, which always counts)."""
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


def _blocks(x, rows):
    """x (R, C) in e4m3 with one float32 scale for `rows` x 128 values: (values, scales)."""
    R, C = x.shape
    r, c = -(-R // rows), -(-C // GROUP)
    a = torch.nn.functional.pad(x, (0, c * GROUP - C, 0, r * rows - R)).view(r, rows, c, GROUP)
    top = a.abs().amax(dim=(1, 3))
    live = top >= TINY
    scale = torch.where(live, top * INV_TOP, 0.0)
    inv = torch.where(live, torch.full_like(top, TOP) / top, 0.0)
    q = (a * inv[:, None, :, None]).clamp_(-TOP, TOP).view(r * rows, c * GROUP)[:R, :C]
    return q.to(E4M3), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    if case["op"] == "logprobs":
        B, n, V, dt = case["seqs"], case["n"], case["V"], DTYPES[case["dtype"]]
        slab = torch.empty(B, n + (1 if case["shifted"] else 0), V, dtype=dt, device="cuda")
        at = torch.log1p(torch.arange(V, device="cuda").float())     # frequent tokens first, as vocabularies are
        for rows in slab.view(-1, V).split(1024):
            rows.copy_(randn(*rows.shape, scale=2.5) - at)
        if case["banned"]:
            slab.masked_fill_(torch.rand(V, device="cuda", generator=g) < 0.3, -math.inf)
        s = {"case": case, "logits": slab[:, :n], "targets": torch.randint(0, V, (B, n), device="cuda", generator=g)}
        mask = torch.ones(B, n, dtype=torch.bool, device="cuda")
        dropped = _masked_rows(n, case["masked"])
        if dropped:
            mask[:, torch.tensor(dropped, device="cuda")] = False
        s["mask"] = mask
        if case["grad"]:  # what the forward pass keeps, and what arrives
            lse, entropy = (torch.zeros(B, n, device="cuda") for _ in range(2))
            for b in range(B):
                for i in range(0, n, 1024):
                    z = s["logits"][b, i:i + 1024].double() / case["T"]
                    l = torch.logsumexp(z, dim=-1)
                    lse[b, i:i + 1024], entropy[b, i:i + 1024] = l.float(), (l - (torch.exp(z - l[:, None]) * z).sum(dim=-1)).float()
            s |= {"lse": torch.where(mask, lse, 0.0), "entropy": torch.where(mask, entropy, 0.0),
                  "grad_logp": randn(B, n), "grad_entropy": randn(B, n, scale=0.1)}
        return s
    if case["op"] == "rms":
        n, H, dt = case["n"], case["H"], DTYPES[case["dtype"]]
        rt = torch.float32 if case["residual"] == "fp32" else dt
        s = {"case": case, "weight": (randn(H, scale=0.2) + 1.0).to(dt)}
        if case["grad"]:  # what the forward pass keeps: the stream it wrote, and 1 / rms
            h = randn(n, H, scale=1.5, dtype=dt if case["residual"] == "none" else rt)
            rstd = (h.double().square().mean(dim=1) + EPS).rsqrt().float()
            return s | {"stream": h, "rstd": rstd, "grad_y": randn(n, H, dtype=dt),
                        "grad_stream": None if case["residual"] == "none" else randn(n, H, dtype=rt)}
        return s | {"x": randn(n, H, dtype=dt), "residual": None if case["residual"] == "none" else randn(n, H, scale=2.0, dtype=rt)}
    if case["op"] == "fp8":
        n, H, V = case["n"], case["H"], case["V"]
        x_q, x_scale = _blocks(randn(n, H), 1)
        w_q, w_scale = _blocks(randn(V, H, scale=2.0 / math.sqrt(H)), GROUP)
        return {"case": case, "x_q": x_q, "x_scale": x_scale, "w_q": w_q, "w_scale": w_scale,
                "bias": randn(V, scale=0.5, dtype=DTYPES[case["dtype"]]) if case["bias"] else None}
    sizes, dt = _sizes(case), DTYPES[case["dtype"]]
    scale = 1.0 if case["inf"] else 4.0 / math.sqrt(sum(sizes))      # norms of about 4
    if case["clip"]:      # views of one packed buffer, as buckets of gradients are
        flat = randn(sum(sizes), scale=scale, dtype=dt)
        return {"case": case, "grads": list(flat.split(sizes)), "flat": flat}
    return {"case": case, "grads": [randn(k, scale=scale, dtype=dt) for k in sizes]}


# ------------------------------------------------------------------------------------------------------- plain forms

def _top(z, k):
    """The k largest values of each row and their places, the lowest index first among equal ones."""
    bits = (z + 0.0).view(torch.int32)                           # + 0.0: -0 and 0 are equal
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64)     # integers in the floats' order
    key = (order << 32) | (0xFFFFFFFF - torch.arange(z.shape[-1], device=z.device))
    index = 0xFFFFFFFF - (torch.topk(key, k, dim=-1).values & 0xFFFFFFFF)
    return z.gather(-1, index), index


def _plain_logprobs(s):
    c, mask, y = s["case"], s["mask"], s["targets"][..., None]
    z = s["logits"].float() * float(np.float32(1.0 / c["T"]))
    if c["grad"]:
        z -= s["lse"][..., None]
        p = z.exp()
        g, h = s["grad_logp"][..., None], s["grad_entropy"][..., None]
        dz = (z.add_(s["entropy"][..., None]).mul_(h).add_(g)).mul_(p).neg_()
        dz.scatter_add_(-1, y, g)
        dz = torch.where(mask[..., None], dz * float(np.float32(1.0 / c["T"])), 0.0)
        return {"grad_logits": dz.to(s["logits"].dtype)}
    out = {}
    if c["top_k"]:
        top, index = _top(z, c["top_k"])
    first = z.amax(dim=-1, keepdim=True)
    at = z.gather(-1, y)[..., 0]
    z -= first
    p = z.exp()
    total = p.sum(dim=-1)
    lse = first[..., 0] + total.log()
    entropy = total.log() - (p * torch.where(p > 0, z, 0.0)).sum(dim=-1) / total
    zero = torch.zeros_like(lse)
    out |= {"logp": torch.where(mask, at - lse, zero), "lse": torch.where(mask, lse, zero),
            "entropy": torch.where(mask, entropy, zero)}
    if c["top_k"]:
        out |= {"top_logp": torch.where(mask[..., None], top - lse[..., None], 0.0),
                "top_index": torch.where(mask[..., None], index, -1)}
    return out


def _plain_rms(s):
    w = s["weight"].float()
    if s["case"]["grad"]:
        h, dy, rstd = s["stream"].float(), s["grad_y"].float(), s["rstd"][:, None]
        hat = h * rstd
        d = dy * w
        dh = (d - hat * (d * hat).mean(dim=1, keepdim=True)) * rstd
        if s["grad_stream"] is not None:
            dh += s["grad_stream"].float()
        return {"grad_stream": dh.to(s["stream"].dtype), "grad_weight": (dy * hat).sum(dim=0).to(s["weight"].dtype)}
    x, out = s["x"], {}
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(s["residual"].dtype)
        out["stream"] = x
    x = x.float()
    rstd = (x.square().mean(dim=1) + EPS).rsqrt()
    y = x * rstd[:, None] * w
    out["rstd"] = rstd
    if s["case"]["fp8"]:
        q, scale = _blocks(y, 1)
        return out | {"q": q, "scale": scale}
    return out | {"y": y.to(s["x"].dtype)}


def _wide(q, scale, rows, dtype):
    return q.to(dtype) * scale.to(dtype).repeat_interleave(rows, dim=0)[:q.shape[0]].repeat_interleave(GROUP, dim=1)[:, :q.shape[1]]


def _plain_fp8(s):
    out = _wide(s["x_q"], s["x_scale"], 1, torch.float32) @ _wide(s["w_q"], s["w_scale"], GROUP, torch.float32).t()
    if s["bias"] is not None:
        out += s["bias"].float()
    return {"out": out.to(DTYPES[s["case"]["dtype"]])}


def _plain_norm(s):
    c, grads = s["case"], s["grads"]
    wide = [g.float() for g in grads]
    if c["inf"]:
        norm = torch.stack([g.abs().amax() for g in wide]).amax()
    else:
        norm = torch.stack([g.square().sum() for g in wide]).sum().sqrt()
    scale = (MAX_NORM / (norm + CLIP_EPS)).clamp(max=1.0)
    if not c["clip"]:
        return {"norm": norm, "scale": scale}
    s["flat"].copy_(s["flat"].float() * scale)
    return {"norm": norm, "grads": s["flat"]}


# ------------------------------------------------------------------------------------------------------- the calls

def run(s):
    if own:
        return _own(s)
    return {"logprobs": _plain_logprobs, "rms": _plain_rms, "fp8": _plain_fp8, "norm": _plain_norm}[s["case"]["op"]](s)


def _own(s):
    import rl_post_loss_amd as rl
    c = s["case"]
    if c["op"] == "logprobs":
        if c["grad"]:
            return {"grad_logits": rl.token_logprobs_bwd(s["logits"], s["targets"], s["mask"], s["lse"], s["entropy"],
                                                         s["grad_logp"], s["grad_entropy"], temperature=c["T"])}
        logp, lse, entropy, top_logp, top_index = rl.token_logprobs_fwd(s["logits"], s["targets"], s["mask"],
                                                                        temperature=c["T"], top_k=c["top_k"])
        out = {"logp": logp, "lse": lse, "entropy": entropy}
        return out | {"top_logp": top_logp, "top_index": top_index} if c["top_k"] else out
    if c["op"] == "rms":
        if c["grad"]:
            dh, dw = rl.rms_norm_bwd(s["grad_y"], s["stream"], s["weight"], s["rstd"], s["grad_stream"])
            return {"grad_stream": dh, "grad_weight": dw}
        if c["fp8"]:
            q, scale, rstd, stream = rl.rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=EPS)
            out = {"q": q, "scale": scale, "rstd": rstd}
        else:
            y, rstd, stream = rl.rms_norm_fwd(s["x"], s["weight"], s["residual"], eps=EPS)
            out = {"y": y, "rstd": rstd}
        return out if stream is None else out | {"stream": stream}
    if c["op"] == "fp8":
        return {"out": rl.fp8_linear(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], s["bias"],
                                     out_dtype=DTYPES[c["dtype"]])}
    kind = math.inf if c["inf"] else 2.0
    if c["clip"]:
        return {"norm": rl.clip_grads(s["grads"], MAX_NORM, norm_type=kind, eps=CLIP_EPS), "grads": s["flat"]}
    norm, scale = rl.grad_norm(s["grads"], max_norm=MAX_NORM, norm_type=kind, eps=CLIP_EPS)
    return {"norm": norm, "scale": scale}


# ------------------------------------------------------------------------------------------------------- the work

def work(case):
    """Bytes: inputs read once (masked rows' logits not at all), outputs written once.  Flops by the formulas' terms."""
    e = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "logprobs":
        n, V = case["seqs"] * case["n"], case["V"]
        valid = case["seqs"] * (case["n"] - len(_masked_rows(case["n"], case["masked"])))
        if case["grad"]:
            return {"bytes": (valid + n) * V * e + n * 25, "flops": 8 * valid * V}
        return {"bytes": valid * V * e + n * (21 + 12 * case["top_k"]), "flops": 7 * valid * V}
    if case["op"] == "rms":
        n, H = case["n"], case["H"]
        r = 4 if case["residual"] == "fp32" else e
        if case["grad"]:
            stream = e if case["residual"] == "none" else r
            b = n * H * (e + 2 * stream + (0 if case["residual"] == "none" else stream)) + 4 * n + 2 * H * e
            return {"bytes": b, "flops": 9 * n * H}
        b = n * H * (e + (0 if case["residual"] == "none" else 2 * r) + (1 if case["fp8"] else e)) + 4 * n + H * e
        return {"bytes": b + (4 * n * -(-H // GROUP) if case["fp8"] else 0), "flops": (8 if case["fp8"] else 5) * n * H}
    if case["op"] == "fp8":
        n, H, V, b = case["n"], case["H"], case["V"], -(-case["H"] // GROUP)
        return {"bytes": n * H + V * H + 4 * b * (n + -(-V // GROUP)) + n * V * e + (V * e if case["bias"] else 0),
                "flops": 2 * n * H * V}
    total = sum(_sizes(case))
    return {"bytes": total * e * (2 if case["clip"] else 1) + 4, "flops": 2 * total}


# ------------------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "rms": _exact_rms, "fp8": _exact_fp8, "norm": _exact_norm}[case["op"]](s)


def _exact_logprobs(s):
    """In groups of rows, so that the logits in 64 bits fit beside the inputs."""
    c, V = s["case"], s["case"]["V"]
    names = ["grad_logits"] if c["grad"] else ["logp", "lse", "entropy"] + (["top_logp"] if c["top_k"] else [])
    parts = {k: [] for k in names}
    for b in range(c["seqs"]):
        for i in range(0, c["n"], 512):
            rows = slice(i, min(i + 512, c["n"]))
            z = torch.div(s["logits"][b, rows].to(torch.float64), c["T"])
            y, on = s["targets"][b, rows], s["mask"][b, rows].to(torch.float64)
            if c["grad"]:
                g, h = s["grad_logp"][b, rows].double()[:, None], s["grad_entropy"][b, rows].double()[:, None]
                logs = z - s["lse"][b, rows].double()[:, None]
                hit = torch.nn.functional.one_hot(y, V).to(torch.float64)
                p = torch.exp(logs)
                d = g * hit - g * p - h * p * (logs + s["entropy"][b, rows].double()[:, None])
                parts["grad_logits"].append((d / c["T"]) * on[:, None])
                continue
            lse = torch.logsumexp(z, dim=1)
            logs = z - lse[:, None]
            p = torch.exp(logs)
            parts["lse"].append(torch.where(on > 0, lse, 0.0))
            parts["logp"].append(torch.where(on > 0, logs[torch.arange(len(y), device=y.device), y], 0.0))
            parts["entropy"].append(-(torch.nan_to_num(p * logs, nan=0.0)).sum(dim=1) * on)
            if c["top_k"]:
                best = torch.sort(logs, dim=1, descending=True).values[:, :c["top_k"]]
                parts["top_logp"].append(torch.where(on[:, None] > 0, best, 0.0))
    shape = (c["seqs"], c["n"])
    out = {k: torch.cat(v).reshape(*shape, *v[0].shape[1:]) for k, v in parts.items()}
    if c["top_k"] and not c["grad"]:
        out["top_index"] = None
    return out


def _exact_rms(s):
    w = s["weight"].to(torch.float64)
    if s["case"]["grad"]:
        h, dy, r = s["stream"].to(torch.float64), s["grad_y"].to(torch.float64), s["rstd"].to(torch.float64)[:, None]
        # d/dh of sum(dy * h * r * w): the row's own term less the one that goes through its mean square
        dh = r * dy * w - (r ** 3 / h.shape[1]) * h * torch.sum(dy * w * h, dim=1, keepdim=True)
        if s["grad_stream"] is not None:
            dh = dh + s["grad_stream"].to(torch.float64)
        return {"grad_stream": dh, "grad_weight": torch.mv((dy * h).t(), r[:, 0])}
    h, out = s["x"].to(torch.float64), {}
    if s["residual"] is not None:      # the norm is that of the stream as it is held
        h = torch.add(h, s["residual"].to(torch.float64))
        out["stream"] = h
        h = h.to(torch.float32).to(s["residual"].dtype).to(torch.float64)
    r = 1.0 / torch.sqrt(torch.sum(h * h, dim=1) / h.shape[1] + EPS)
    y = w * (h * r[:, None])
    out["rstd"] = r
    if not s["case"]["fp8"]:
        return out | {"y": y}
    n, H = y.shape
    groups = torch.nn.functional.pad(y, (0, -H % GROUP)).reshape(n, -1, GROUP)
    scale = groups.abs().amax(dim=2) / TOP
    q = groups / torch.where(scale > 0, scale, 1.0)[..., None]
    return out | {"q": q.reshape(n, -1)[:, :H], "scale": scale}


def _exact_fp8(s):
    x, w = _wide(s["x_q"], s["x_scale"], 1, torch.float64), _wide(s["w_q"], s["w_scale"], GROUP, torch.float64)
    out = torch.empty(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for i in range(0, w.shape[0], 16384):
        out[:, i:i + 16384] = torch.matmul(x, w[i:i + 16384].t().contiguous())
    return {"out": out if s["bias"] is None else out + s["bias"].to(torch.float64)}


def _exact_norm(s):
    c = s["case"]
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        d = g.to(torch.float64)
        total = torch.maximum(total, d.abs().max()) if c["inf"] else total + torch.dot(d, d)
    norm = total if c["inf"] else torch.sqrt(total)
    scale = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + CLIP_EPS))
    return {"norm": norm, "grads": s["flat"].to(torch.float64) * scale} if c["clip"] else {"norm": norm, "scale": scale}
