"""Token log-probabilities: rows of NaN write all of their results, NaN and indices of -1, along every path.

Through the C entry, with the outputs filled beforehand, so that what is not written shows.
"""
import pytest
import torch

import rl_post_loss_amd as rl
from test_token_logprobs import DEV, DT, forward_case, make

pytestmark = pytest.mark.gpu
BITS = {"bf16": (torch.int16, 0x7FC0), "fp16": (torch.int16, 0x7E00), "fp32": (torch.int32, 0x7FC00000)}
STALE = 12345


def nan_of(V, dtype, negative):
    kind, bits = BITS[dtype]
    sign = torch.iinfo(kind).min if negative else 0
    return torch.full((V,), bits + sign, dtype=kind).view(DT[dtype])


def bad_rows(V, dtype, top_k):
    """Rows that have no distribution: NaN alone, of either sign, beside fewer or more than top_k others, beside an infinity."""
    g = torch.Generator().manual_seed(V)
    rows = []
    for negative in (False, True):
        row = nan_of(V, dtype, negative)
        rows.append(row)
        for others in (1, top_k - 1, top_k + 1):
            some = row.clone()
            some[torch.randperm(V, generator=g)[:others]] = 1.5
            rows.append(some)
        ends = row.clone()
        ends[0], ends[-1] = float("inf"), float("-inf")
        rows.append(ends)
        one = torch.randn(V, generator=g).to(DT[dtype])
        one[V // 2] = row[0]
        rows.append(one)
    return torch.stack(rows)


def through_the_c_entry(z, y, top_k):
    rows, V = z.shape
    lib = rl.library()
    z, y = z.to(DEV), y.to(DEV)
    logp, lse, entropy = (torch.full((rows,), float(STALE), device=DEV) for _ in range(3))
    top = torch.full((rows, top_k), float(STALE), device=DEV)
    index = torch.full((rows, top_k), STALE, dtype=torch.int64, device=DEV)
    nbytes = lib.token_logprobs_workspace_bytes(rows, V, top_k)
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=DEV)
    at = (ws.data_ptr() + 255) // 256 * 256
    status = lib.token_logprobs_fwd(z.data_ptr(), y.data_ptr(), None, rows, V, rows, 0, V, rl.DTYPE[z.dtype], 1.0, top_k,
                                    logp.data_ptr(), lse.data_ptr(), entropy.data_ptr(), top.data_ptr(), index.data_ptr(), at, nbytes,
                                    torch.cuda.current_stream().cuda_stream)
    assert status == 0
    return logp, lse, entropy, top, index


# rows in pieces (each of which has more candidates than there is room for in 16 bits), whole rows, rows of a wavefront
@pytest.mark.parametrize("rows,V,dtype,top_k", [(8, 128256, "bf16", 20), (8, 128256, "bf16", 64), (8, 128256, "fp16", 5),
                                                (8, 128256, "fp32", 20), (1, 150001, "bf16", 64), (33, 70001, "bf16", 64),
                                                (64, 128256, "bf16", 20), (2, 1 << 22, "bf16", 64), (1030, 40000, "bf16", 20),
                                                (20, 40000, "fp16", 64), (20, 4097, "fp32", 64), (40, 4096, "bf16", 64),
                                                (40, 1000, "fp32", 20), (40, 100, "fp16", 64)])
def test_all_results_of_rows_without_a_distribution_are_written(rows, V, dtype, top_k):
    bad = bad_rows(V, dtype, top_k)
    z, y, _ = make(rows, V, dtype, seed=3)
    at = range(0, len(bad), max(1, rows - 1)) if rows > 1 else range(len(bad))
    for first in at:                                           # all but the last row of a call
        some = bad[first:first + max(1, rows - 1)]
        n = len(some)
        w = z.clone()
        w[:n] = some
        logp, lse, entropy, top, index = through_the_c_entry(w, y, top_k)
        for name, t in (("logp", logp), ("lse", lse), ("entropy", entropy), ("top_logp", top)):
            assert t[:n].isnan().all(), (name, first, (~t[:n].isnan()).nonzero()[:3].tolist())
        assert (index[:n] == -1).all(), (first, index[:n][index[:n] != -1][:3])
        if rows > n and V <= 200000:
            last = slice(max(n, rows - 2), rows)
            forward_case(w[last], y[last], 1.0, [t[last] for t in (logp, lse, entropy, top, index)], top_k)
