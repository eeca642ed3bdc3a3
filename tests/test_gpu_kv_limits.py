"""The key-value side at the ends of what it takes."""
import math

import pytest
import torch

from dspark_draft_sampling_gb300 import api

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# ---- many keys, each far below the largest -------------------------------------------------
@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weights_far_below_the_largest_add_up(dtype, n):
    """Two keys (of the first two tiles of 128) weigh 1, 65,998 others 2^-25.2 each and bring the whole output, 8.5e-4.

    Tolerance: the output's rounding and each weight's (u relative, twice), a weight's spacing where it is smallest (2^-31 of the
    running maximum, so 2^-32 a key), 2^-16 relative for the score, whose fp32 error is 2^-24 of 25; twice their sum."""
    keys, heads, seqs, dim, page = 66000, 8, 19, 64, 128
    pages = -(-keys // page)
    pool = torch.zeros((pages, 1, 2, heads, page, dim), dtype=dtype, device="cuda")
    big, per_dim = 8.734375 if dtype == F16 else 8.75, 1.0 + torch.arange(dim, dtype=torch.float64) / 64  # exact in the type
    pool[:, 0, 1] = per_dim.to(dtype).cuda()
    for p in (0, 128 // page):
        pool[p, 0, 0, :, 0, 0] = big
        pool[p, 0, 1, :, 0] = 0.0
    # rows that share all pages: whole rows for each SM, as many as there are
    table = torch.arange(pages, dtype=torch.int32).expand(seqs, pages).contiguous().cuda()
    cache = api.PagedCache(pool, table, ints([keys] * seqs), ints([seqs] * pages))
    q = torch.zeros((seqs * n, heads, dim), dtype=dtype, device="cuda")
    q[:, :, 0] = 16.0
    out, lse = api.paged_attention(q, cache, 0, ints(range(0, seqs * n + 1, n)), max_new=n, causal=False, return_lse=True)
    assert cache.status() == 0
    top = 16.0 * big / 8.0
    mass = (keys - 2) * math.exp(-top)
    want = mass / (2.0 + mass) * per_dim
    u = 2.0**-11 if dtype == F16 else 2.0**-8
    tol = 2 * ((2 * u + 2.0**-16) * want + keys * 2.0**-32 * per_dim)
    assert ((out.cpu().double() - want).abs() <= tol).all(), (float(out.max()), float(want.max()))
    assert ((lse.cpu().double() - (top + math.log(2.0 + mass))).abs() <= 2 * 2.0**-20 * (1 + top)).all()

