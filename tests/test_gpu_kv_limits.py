"""The key-value side at the ends of what it takes."""
import math

import pytest
import torch

from dspark_draft_sampling_gb300 import api

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
HEADER, COUNTERS, TIMEOUT = api.CACHE_HEADER_BYTES, 256, 2  # bytes of the workspace's header, its arrival counts, a status bit


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def filled_cache(lens, *, kv_heads, dim, dtype, page=16, seed=0):
    wide = max(1, max(-(-n // page) for n in lens))
    cache = api.PagedCache.empty(len(lens) * wide + 1, len(lens), wide, layers=1, kv_heads=kv_heads, page_size=page, head_dim=dim,
                                 dtype=dtype)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cache.pool.copy_(torch.randn(cache.pool.shape, generator=gen, device="cuda"))
    cache.extend(ints(range(len(lens))), ints(lens))
    return cache


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


# ---- what a wait that gave up leaves behind -----------------------------------------------
@pytest.mark.parametrize("n", [1, 40])
def test_status_after_a_wait_that_gave_up_makes_the_workspace_whole(n):
    # such a call can end between the arrivals of a cut item's blocks; here they are written as it may leave them
    cache = filled_cache([9000], kv_heads=1, dim=128, dtype=BF16, page=64)
    q = torch.randn((n, 4, 128), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    cu = ints([0, n])
    want = api.paged_attention(q, cache, 0, cu)
    assert cache.status() == 0
    cache.workspace[COUNTERS:HEADER].fill_(1)
    cache.workspace[0] = TIMEOUT
    assert cache.status() == api.DSPARK_ERR_TIMEOUT
    cache.workspace[HEADER:].fill_(255)  # partial sums of earlier calls are no answer
    for _ in range(2):
        assert torch.equal(api.paged_attention(q, cache, 0, cu), want)
    assert cache.status() == 0 and not cache.workspace[:HEADER].any()


# ---- windows without an end ----------------------------------------------------------------
@pytest.mark.parametrize("window", [2**30, 2**31 - 1])
@pytest.mark.parametrize("causal", [True, False])
def test_a_window_longer_than_any_row_hides_nothing(causal, window):
    # also where a chunk is longer than its row, so that positions are negative
    cache = filled_cache([40, 300, 3], kv_heads=1, dim=64, dtype=F16)
    q = torch.randn((340, 2, 64), generator=torch.Generator().manual_seed(3)).half().cuda()
    cu = ints([0, 50, 150, 340])
    want, want_lse = api.paged_attention(q, cache, 0, cu, causal=causal, return_lse=True)
    got, lse = api.paged_attention(q, cache, 0, cu, causal=causal, window=window, return_lse=True)
    assert cache.status() == 0
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


# ---- axes of one entry ---------------------------------------------------------------------
def test_strides_of_axes_of_one_entry_do_not_matter():
    # one token, or one head, whose stride is whatever the tensor was made by: it is never used
    gen = torch.Generator().manual_seed(2)
    turns = api.RotaryTable(api.rotary_frequencies(64))
    token = torch.randn((4, 64, 1), generator=gen).half().cuda().permute(2, 0, 1)  # [1, 4, 64], strides (1, 64, 1)
    head = torch.randn((3, 64, 1), generator=gen).half().cuda().permute(0, 2, 1)   # [3, 1, 64], strides (64, 1, 1)
    for x in (token, head):
        pos = ints(range(7, 7 + x.shape[0]))
        assert torch.equal(api.rotary(x, pos, turns), api.rotary(x.clone(memory_format=torch.contiguous_format), pos, turns))
    for q, kv in ((token, token[:, :1]), (token, token[:, :2]), (head, head)):
        n, got = q.shape[0], []
        for dense in (False, True):
            cache = filled_cache([20 + n], kv_heads=kv.shape[1], dim=64, dtype=F16)
            a, b = (x.clone(memory_format=torch.contiguous_format) if dense else x for x in (q, kv))
            turned = api.rotary_append(a, b, b, cache, 0, ints([0, n]), turns)
            got.append((turned, cache.pool, api.paged_attention(a, cache, 0, ints([0, n])),
                        api.paged_attention(a, cache, 0, ints([0, n]), out=torch.empty_like(a))))
            assert cache.status() == 0
        for x, y in zip(*got):
            assert torch.equal(x, y)
