"""The lse^2 penalty at its largest: the gradient's factor 1 + 2 z_loss lse in fp16.

Tolerances are those of tests/test_linear_cross_entropy.py; with z_loss over 0.254 dz is held at 128 or 64 times its value
in fp16, so its absolute rounding below the normal range is 2^-25 over that.
"""
import pytest
import torch

import rl_post_loss_amd as rl
from test_linear_cross_entropy import E, SUB, U, check, expected, make, on_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shift", [130.0, 480.0, -480.0])
@pytest.mark.parametrize("z_loss", [0.25, 0.26, 0.5, 0.51, 1.0])
def test_large_penalties_of_large_logits(z_loss, shift, dtype):
    for n, H, V in ((70, 64, 300), (1100, 40, 1500)):
        c = make(n, H, V, dtype, ignored=0.2, seed=3)
        c["b"] = (c["b"].float() + shift).to(c["b"].dtype)
        args = on_device(c)
        out = rl.linear_cross_entropy(*args, z_loss=z_loss)
        want = expected(c, z_loss)
        check("loss", out[0], want["loss"])
        keep = c["y"] != -100
        s = 1.0 / int(keep.sum())
        more = s * SUB[dtype] / 64.0                  # of one element of dz
        h, w = c["h"].double().abs()[keep], c["w"].double().abs()
        value, tol = want["grad_hidden"]
        tol = tol + more * w.sum(0) * keep[:, None]
        check("grad_hidden", out[1], (value, tol), U[dtype], SUB[dtype])
        value, tol = want["grad_weight"]
        check("grad_weight", out[2], (value, tol + more * h.sum(0)), U[dtype], SUB[dtype])
        value, tol = want["grad_bias"]
        check("grad_bias", out[3], (value, tol), U[dtype], SUB[dtype])
