"""The AdamW step of the library in numpy: each operation one IEEE float32 operation in the order the C header's
formulas give, with the 8-bit moments' blocks, random bits and rounding written out element by element in arrays."""
import math

import numpy as np

f32 = np.float32
BLOCK = 256


def mix(x):
    x = np.asarray(x, dtype=np.uint64) & np.uint64(0xFFFFFFFF)
    for shift, factor in ((16, 0x85EBCA6B), (13, 0xC2B2AE35)):
        x = x ^ (x >> np.uint64(shift))
        x = (x * np.uint64(factor)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def random_words(seed, step, tensor, n, start=0):
    """The words of elements start .. start + n (which share their upper 32 bits)."""
    key = mix(mix(mix(seed) ^ np.uint64(step & 0xFFFFFFFF)) ^ np.uint64(tensor))
    i = np.arange(n, dtype=np.uint64) + np.uint64(start)
    return mix((i & np.uint64(0xFFFFFFFF)) ^ mix(key + (i >> np.uint64(32))))


E4M3 = np.array([s * ((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) if (e, m) != (15, 7) else np.nan
                 for s in (1, -1) for e in range(16) for m in range(8)], dtype=np.float32)   # value of each byte


def decode(codes, scale):
    with np.errstate(invalid="ignore"):
        return E4M3[codes] * np.repeat(scale, BLOCK)[:codes.size]


def encode(x, words16, root):
    """(bytes, scales) of float32 x: rounded up where the fraction below the last place plus words16 / 2^16 reaches 1."""
    n = x.size
    a = np.zeros((n + BLOCK - 1) // BLOCK * BLOCK, dtype=np.float32)
    a[:n] = np.abs(x)
    a = a.reshape(-1, BLOCK)
    ok = np.isfinite(a)
    top = np.where(ok, a, 0).max(axis=1).astype(np.float32)
    live = top >= f32(2.0 ** -118)
    with np.errstate(all="ignore"):
        scale = np.where(live, top * (f32(1) / f32(448)), f32(0)).astype(np.float32)
        inv = np.where(live, f32(448) / top, f32(0)).astype(np.float32)
        q = (a * inv[:, None]).reshape(-1)[:n]
        good = np.isfinite(x)
        q = np.where(good, q, f32(0))
        e = np.maximum(np.floor(np.log2(np.maximum(q, f32(1e-30)).astype(np.float64))).astype(int), -6)
        step = np.exp2(e - 3.0)
        t = (q / step).astype(np.float32) + words16.astype(np.float32) * f32(2.0 ** -16)
        v = np.minimum(np.floor(t) * step, 448.0)
    if root:
        v = np.where((x > 0) & good, np.maximum(v, 2.0 ** -9), v)
    positive = E4M3[:127].astype(np.float64)
    code = np.searchsorted(positive, v)
    assert np.array_equal(positive[code], v), "a rounded value is not an e4m3 value"
    code = np.where(x < 0, code + 128, code)
    return np.where(good, code, 127).astype(np.uint8), scale


def coefficients(lr, betas, eps, step):
    b1, b2 = betas
    return dict(b1=f32(b1), b2=f32(b2), c1=f32(1 - b1), c2=f32(1 - b2), eps=f32(eps), size=f32(lr / (1 - b1 ** step)),
                root=f32(1 / math.sqrt(1 - b2 ** step)), lr=lr)


def step(p, g, m, v, k, weight_decay):
    """(p, m, sqrt(v), v) after one step, all float32; v the second moment."""
    with np.errstate(all="ignore"):
        m = m * k["b1"] + g * k["c1"]
        v = v * k["b2"] + (g * k["c2"]) * g
        r = np.sqrt(v)
        u = (m / (r * k["root"] + k["eps"])) * k["size"]
        p = p * f32(1 - k["lr"] * weight_decay) - u
    return p, m, r, v
