"""Products of 8-bit operands with an outlier column beside small ones: what the public header says of both kinds of outputs.

x has one large value in each block, w small ones, so that a row's result is the sum of many small products beside a large one that
cancels against another block's.  eps = 2^-24.  float32 outputs: the sums' order alone, (2 * 128 + H / 128 + 8) eps sum |x w| s.
16-bit outputs: 7 * 2^-13 of the largest product of each aligned eight more, and half a step of the output; and
the small products that share an eight with the outlier are seen to be lost there, since the bound would otherwise say nothing.
"""
import pytest
import torch

import rl_post_loss_amd as rl
from test_fp8_linear import DEV, E32, dropped, wide

pytestmark = pytest.mark.gpu


def operands(n, H, V):
    """Blocks in pairs: outlier 256 in column 3, against weights of 256 and -256, and 1 elsewhere; weights of 12 beside them."""
    x, w = torch.ones(n, H), torch.full((V, H), 12.0)
    for k in range(0, H, 128):
        x[:, k + 3] = 256.0
        w[:, k + 3] = 256.0 if k // 128 % 2 == 0 else -256.0
    w[::2, 5] = 4.0
    f8 = torch.float8_e4m3fn
    return x.to(f8), torch.ones(n, -(-H // 128)), w.to(f8), torch.ones(-(-V // 128), -(-H // 128))


# few rows, 64 x 64, K shared, 128 x 64, 128 x 128, 256 x 256
@pytest.mark.parametrize("n,H,V", [(3, 512, 300), (40, 512, 20000), (64, 2048, 700), (128, 2048, 50001), (700, 1024, 8000),
                                   (1100, 512, 40000)])
def test_small_products_beside_an_outlier(n, H, V):
    d = [t.to(DEV) for t in operands(n, H, V)]
    rows, cols = torch.tensor([0, n - 1]), torch.tensor([0, 1, 127, 128, V - 2, V - 1])
    take = lambda t, i: t.view(torch.uint8)[i].view(t.dtype)  # noqa: E731
    a = wide(take(d[0].cpu(), rows), d[1].cpu()[rows], 1)
    b = wide(take(d[2].cpu(), cols), d[3].cpu().repeat_interleave(128, 0)[cols], 1)
    want = a @ b.t()
    order = (256 + H / 128 + 8) * E32 * (a.abs() @ b.abs().t())
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        out = rl.fp8_linear(*d, out_dtype=dtype)[rows.to(DEV)][:, cols.to(DEV)].cpu().double()
        tol = order
        if dtype != torch.float32:
            tol = tol + dropped(a, b) + torch.finfo(dtype).eps / 2 * (want.abs() + dropped(a, b))
            assert ((out - want).abs() > order + torch.finfo(dtype).eps / 2 * want.abs()).any()
        assert ((out - want).abs() <= tol).all(), (dtype, (out - want).abs().max(), tol.min())
