"""Attention over the paged cache against a 64-bit reference, at the sizes and masks where it can go wrong.

Tolerance of an output, from the number formats: the result is rounded once (unit roundoff u of its type), the
weights are rounded to the same type before they multiply the values (u relative to sum w|v|; in fp16 also
2^-24 absolute a weight, relative to the largest), and the scores carry fp32 errors of at most head_dim * 2^-24
* sum|q k| * scale, which the weights inherit as relative errors.  Twice the sum of these is allowed.  The log-sum
carries the scores' error and 2^-20 relative of its own."""
import math

import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def make_cache(gen, lens, *, dtype, dim, kv_heads, page, layers=1, spare=3, rows=None, poison=True):
    """Rows of the given lengths on shuffled pages; what no row can see is NaN."""
    count = [-(-n // page) for n in lens]
    wide = max(1, max(count)) + 1
    pages = sum(count) + spare
    pool = torch.randn((pages, layers, 2, kv_heads, page, dim), generator=gen).to(dtype)
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(lens), wide), -1, dtype=torch.int32)
    seen = torch.zeros((pages, page), dtype=torch.bool)
    for r, n in enumerate(lens):
        for j in range(count[r]):
            p = order.pop()
            table[r, j] = p
            seen[p, : min(page, n - j * page)] = True
    if poison:
        pool.permute(0, 4, 1, 2, 3, 5)[~seen] = math.nan
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    cuda = [t.cuda() for t in (pool, table, torch.tensor(lens, dtype=torch.int32), refs)]
    return api.PagedCache(*cuda), pool, table


def check(case, *, seed=0, strided=False, rows=None, layer=0, layers=1, q_gain=1.0, max_new=None, stream=None):
    dtype, dim, q_heads, kv_heads, page, seqs, causal, window = case
    gen = torch.Generator().manual_seed(seed)
    lens = [n for _, n in seqs]
    table_lens = lens if rows is None else [lens[rows.index(r)] for r in range(len(lens))]
    cache, pool, table = make_cache(gen, table_lens, dtype=dtype, dim=dim, kv_heads=kv_heads, page=page, layers=layers)
    cu = [0]
    for n, _ in seqs:
        cu.append(cu[-1] + n)
    q = (torch.randn((cu[-1], q_heads, dim), generator=gen) * q_gain).to(dtype)
    scale = 1.0 / math.sqrt(dim)
    kw = dict(causal=causal, window=window, max_new=max_new, return_lse=True,
              rows=None if rows is None else torch.tensor(rows, dtype=torch.int32).cuda())
    cu_t = torch.tensor(cu, dtype=torch.int32).cuda()
    if strided:  # a slice of a fused projection, and an output with room between its tokens
        fused = torch.full((cu[-1], q_heads + 2 * kv_heads, dim), math.nan, dtype=dtype, device="cuda")
        fused[:, :q_heads] = q.cuda()
        out = torch.full((cu[-1], q_heads + 1, dim), 7.0, dtype=dtype, device="cuda")
        got, lse = api.paged_attention(fused[:, :q_heads], cache, layer, cu_t, out=out[:, :q_heads], **kw)
        torch.cuda.synchronize()
        assert (out[:, q_heads] == 7.0).all()
    else:
        got, lse = api.paged_attention(q.cuda(), cache, layer, cu_t, **kw)
    assert cache.status() == 0
    u = ref.UNIT[dtype]
    for s, (n, length) in enumerate(seqs):
        row = s if rows is None else rows[s]
        k, v = ref.row_tokens(pool, table, layer, row, length)
        want, want_lse, w_abs, p_abs, dots = ref.attention(q[cu[s] : cu[s + 1]].double(), k, v, n, causal=causal,
                                                           window=window, scale=scale)
        score_err = dim * 2.0**-24 * dots
        tol = u * want.abs() + (u + 2 * score_err + 2.0**-20) * w_abs + (2.0**-24 if dtype == F16 else 0.0) * (1 + p_abs)
        err = (got[cu[s] : cu[s + 1]].cpu().double() - want).abs()
        assert (err <= 2 * tol).all(), (s, float(err.max()), float((err / (tol + 1e-30)).max()))
        have = lse[cu[s] : cu[s + 1]].cpu().double()
        empty = want_lse == -math.inf
        assert (have[empty] == -math.inf).all() and (got[cu[s] : cu[s + 1]].cpu()[empty] == 0).all()
        assert ((have - want_lse)[~empty].abs() <= 2 * (score_err + 2.0**-20 * (1 + want_lse[~empty].abs()))).all()


CASES = {
    # dtype, head_dim, q_heads, kv_heads, page, [(new, length)], causal, window
    "one_token_one_key": (BF16, 128, 4, 1, 16, [(1, 1)], True, 0),
    "one_token": (F16, 64, 8, 2, 16, [(1, 130)], True, 0),
    "tile_edges": (BF16, 128, 2, 2, 16, [(1, 127), (1, 128), (1, 129), (1, 255), (1, 256), (1, 257)], True, 0),
    "page_edges": (F16, 128, 4, 2, 32, [(3, 31), (3, 32), (3, 33), (2, 2), (5, 65)], True, 0),
    "empty_rows": (BF16, 64, 4, 4, 16, [(0, 0), (2, 0), (3, 1), (0, 40), (1, 17), (5, 3)], True, 0),
    "empty_rows_full": (BF16, 64, 4, 4, 16, [(2, 0), (3, 1), (1, 17)], False, 0),
    "draft_block": (BF16, 128, 32, 8, 16, [(7, 300), (7, 7), (7, 1025), (7, 64)], False, 0),
    "verify": (F16, 128, 16, 2, 64, [(8, 700), (1, 1400), (5, 129)], True, 0),
    "window": (BF16, 64, 6, 2, 16, [(9, 400), (40, 40), (1, 3), (33, 161)], True, 17),
    "window_one": (F16, 64, 2, 1, 16, [(5, 50)], True, 1),
    "window_full": (F16, 128, 3, 1, 16, [(20, 300)], False, 100),
    "odd_group": (F16, 64, 7, 1, 32, [(37, 290), (100, 100)], True, 0),
    "group_of_12": (BF16, 128, 12, 1, 16, [(23, 200)], True, 0),
    "group_of_128": (BF16, 64, 128, 1, 16, [(3, 200)], True, 0),
    "chunk": (BF16, 128, 4, 1, 128, [(150, 411)], True, 0),
    "chunk_no_group": (F16, 128, 2, 2, 256, [(300, 300), (129, 600)], True, 0),
    "prompt": (BF16, 64, 2, 1, 64, [(515, 515)], True, 0),
    "many": (F16, 64, 2, 1, 16, [(1 + i % 3, 1 + 37 * i % 211) for i in range(70)], True, 0),
    "split_long": (BF16, 128, 4, 1, 64, [(1, 9000)], True, 0),
    "split_ragged": (F16, 128, 2, 1, 16, [(2, 5001), (1, 16), (4, 2500)], True, 0),
    # cut into so many parts that they are joined in two steps
    "split_chunk": (BF16, 128, 4, 1, 64, [(32, 9000)], True, 0),
    "split_pairs": (F16, 128, 3, 1, 128, [(49, 8720)] * 3, True, 0),
    "split_pairs_one_row": (BF16, 64, 4, 1, 32, [(33, 12001)], False, 0),
    "split_window": (F16, 64, 8, 2, 16, [(60, 7000), (1, 300)], True, 3000),
    # no more query tiles than SMs: a block to each, the last ones with nothing to do
    "whole_items": (BF16, 64, 8, 2, 16, [(130, 130), (0, 9), (257, 300), (1, 1), (70, 0), (64, 900)], True, 0),
    "whole_items_window": (F16, 128, 4, 4, 32, [(200, 700), (90, 90)], True, 50),
    "whole_items_tokens": (F16, 128, 4, 2, 64, [(1, 900), (1, 1000), (1, 700), (0, 0), (1, 950)], True, 0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name):
    case = list(CASES[name])
    # a chunk longer than its row: the positions before the row's start see nothing
    check(tuple(case), seed=len(name))


@pytest.mark.parametrize("name", ["draft_block", "window", "chunk_no_group", "odd_group"])
def test_strided_queries_and_output(name):
    check(CASES[name], seed=5, strided=True)


def test_rows_and_layers():
    check((BF16, 128, 4, 2, 16, [(3, 70), (1, 200), (9, 9)], True, 0), rows=[2, 0, 1], layers=3, layer=1, seed=6)


@pytest.mark.parametrize("max_new", [1, 7, 4000])
def test_the_hint_only_costs_time(max_new):
    check((F16, 64, 4, 2, 16, [(70, 300), (1, 40), (130, 131)], True, 0), max_new=max_new, seed=7)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_peaked_scores(dtype):
    # scores far apart, so that the running maximum rises many times and most weights vanish
    check((dtype, 128, 4, 1, 16, [(5, 700), (1, 2000)], True, 0), q_gain=20.0, seed=8)


def test_same_bits_twice_and_on_another_stream():
    gen = torch.Generator().manual_seed(9)
    cache, _, _ = make_cache(gen, [3001, 50, 777], dtype=BF16, dim=128, kv_heads=2, page=16)
    q = torch.randn((6, 8, 128), generator=gen).to(BF16).cuda()
    cu = torch.tensor([0, 1, 5, 6], dtype=torch.int32).cuda()
    first = api.paged_attention(q, cache, 0, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.empty_like(first) for _ in range(4)]
    for o in outs:
        api.paged_attention(q, cache, 0, cu, out=o, stream=side)
    side.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), first.view(torch.int16))


def test_in_a_graph_with_lengths_that_change():
    gen = torch.Generator().manual_seed(10)
    cache, pool, table = make_cache(gen, [600], dtype=BF16, dim=64, kv_heads=1, page=16, poison=False)
    q = torch.randn((1, 2, 64), generator=gen).to(BF16).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    api.paged_attention(q, cache, 0, cu, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_attention(q, cache, 0, cu, out=out)
    for length in (600, 1, 129, 300):
        cache.length.fill_(length)
        graph.replay()
        torch.cuda.synchronize()
        k, v = ref.row_tokens(pool, table, 0, 0, length)
        want, _, w_abs, _, _ = ref.attention(q.cpu().double(), k, v, 1, causal=True, window=0, scale=0.125)
        assert ((out.cpu().double() - want).abs() <= 2 * (2.0**-8 * (want.abs() + w_abs) + 1e-4 * w_abs)).all()


def test_bad_indices_are_recorded():
    gen = torch.Generator().manual_seed(11)
    cache, _, _ = make_cache(gen, [100, 40], dtype=F16, dim=64, kv_heads=1, page=16, poison=False)
    q = torch.randn((2, 2, 64), generator=gen).to(F16).cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    good = api.paged_attention(q, cache, 0, cu)
    assert cache.status() == 0
    rows = torch.tensor([0, 9], dtype=torch.int32).cuda()
    got, lse = api.paged_attention(q, cache, 0, cu, rows=rows, return_lse=True)
    assert cache.status() == api.DSPARK_ERR_INDEX
    assert torch.equal(got[0], good[0]) and (got[1] == 0).all() and (lse[1] == -math.inf).all()
    cache.table[1, 1] = 1 << 20
    got = api.paged_attention(q, cache, 0, cu)
    assert cache.status() == api.DSPARK_ERR_INDEX and torch.equal(got[0], good[0]) and got.isfinite().all()
    assert cache.status() == 0  # reported once


def test_refusals():
    cache = api.PagedCache.empty(8, 2, 4, layers=2, kv_heads=2, page_size=16, head_dim=64, dtype=F16)
    q = torch.zeros((3, 4, 64), dtype=F16, device="cuda")
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")

    def refused(status, *a, **kw):
        with pytest.raises(api.DsparkError) as e:
            api.paged_attention(*a, **kw)
        assert e.value.status == status

    refused(api.DSPARK_ERR_INVALID, q, cache, 2, cu)
    refused(api.DSPARK_ERR_INVALID, q, cache, -1, cu)
    refused(api.DSPARK_ERR_INVALID, q[:, :3], cache, 0, cu)
    refused(api.DSPARK_ERR_INVALID, q, cache, 0, cu, window=-1)
    refused(api.DSPARK_ERR_UNSUPPORTED, torch.zeros((1, 260, 64), dtype=F16, device="cuda"), cache, 0, cu)
    wide = torch.zeros((3, 4, 68), dtype=F16, device="cuda")
    refused(api.DSPARK_ERR_INVALID, wide[:, :, 4:], cache, 0, cu)
    for bad in (q.to(BF16), q[0], q.cpu(), q[..., :32], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            api.paged_attention(bad, cache, 0, cu)
    with pytest.raises(ValueError):
        api.paged_attention(q, cache, 0, cu.long())
    with pytest.raises(ValueError):
        api.paged_attention(q, cache, 0, cu, out=q[:2])
    # nothing to do is no error
    assert api.paged_attention(q[:0], cache, 0, cu).shape == (0, 4, 64)
    assert cache.status() == 0


@pytest.mark.parametrize("n", [3, 200])
def test_a_wait_that_gave_up_is_reported(n):
    # every softmax thread first waits 20 ms on a barrier that nothing signals; the results are whole all the same
    gen = torch.Generator().manual_seed(12)
    cache, _, _ = make_cache(gen, [700], dtype=BF16, dim=128, kv_heads=1, page=16)
    q = torch.randn((n, 4, 128), generator=gen).to(BF16).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    want = api.paged_attention(q, cache, 0, cu)
    assert cache.status() == 0
    got = torch.empty_like(want)
    lib = api.load_library()
    args = api._ATTENTION_ARGS.pack(q.data_ptr(), got.data_ptr(), 0, 0, cu.data_ptr(), 512, 128, 512, 128, 0, n, 4, 1, n, 1, 0,
                                    128 ** -0.5)
    status = lib.dspark_paged_attention_debug(cache._ref, args, 20000, torch.cuda.current_stream().cuda_stream)
    assert status == 0 and cache.status() == api.DSPARK_ERR_TIMEOUT
    assert torch.equal(got, want)
    assert torch.equal(api.paged_attention(q, cache, 0, cu), want) and cache.status() == 0


@pytest.mark.parametrize("causal", [True, False])
def test_pages_before_the_window_may_be_gone(causal):
    # what no token of the chunk sees is NaN, and the table entries of whole pages before the window point nowhere
    gen = torch.Generator().manual_seed(13)
    n, window, lens = 5, 100, [400, 131, 90]
    cache, pool, table = make_cache(gen, lens, dtype=F16, dim=64, kv_heads=1, page=16)
    q = torch.randn((n * 3, 2, 64), generator=gen).to(F16).cuda()
    cu = torch.tensor([0, n, 2 * n, 3 * n], dtype=torch.int32).cuda()
    first = [max(0, length - n - window + 1) for length in lens]
    clean = pool.clone()
    for r, f in enumerate(first):
        for p in range(f):
            pool[table[r, p // 16], :, :, :, p % 16] = math.nan
    cache.pool.copy_(pool)
    gone = cache.table.clone()
    for r, f in enumerate(first):
        gone[r, : f // 16] = torch.tensor([-1, 10**6, -(2**31)] * 10, dtype=torch.int32)[: f // 16].cuda()
    cache.table.copy_(gone)
    got = api.paged_attention(q, cache, 0, cu, causal=causal, window=window)
    assert cache.status() == 0
    for s, length in enumerate(lens):
        k, v = ref.row_tokens(clean, table, 0, s, length)
        want, _, w_abs, p_abs, dots = ref.attention(q[s * n:(s + 1) * n].cpu().double(), k, v, n, causal=causal, window=window, scale=0.125)
        tol = 2.0**-11 * want.abs() + (2.0**-11 + 2 * 64 * 2.0**-24 * dots + 2.0**-20) * w_abs + 2.0**-24 * (1 + p_abs)
        assert ((got[s * n:(s + 1) * n].cpu().double() - want).abs() <= 2 * tol).all()


def test_outputs_belong_to_the_stream_that_writes_them():
    gen = torch.Generator().manual_seed(14)
    cache, _, _ = make_cache(gen, [3000], dtype=BF16, dim=128, kv_heads=2, page=16)
    q = torch.randn((4, 8, 128), generator=gen).to(BF16).cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32).cuda()
    want = api.paged_attention(q, cache, 0, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):  # outputs dropped at once: their memory may only be taken up again on the same stream
        got, _ = api.paged_attention(q, cache, 0, cu, return_lse=True, stream=side)
        trash = torch.full_like(q, float("nan"))
        del trash
    side.synchronize()
    assert torch.equal(got, want)
