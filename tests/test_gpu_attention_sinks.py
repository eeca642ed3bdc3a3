"""Attention over the paged cache with a window and a row's first tokens that stay visible, against 64 bits.

The tolerance is that of test_gpu_paged_attention.  Whatever no token of a chunk sees is NaN, behind a row's end as well as between its
first tokens and the window, and table entries of pages that hold nothing else point nowhere."""
import math

import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests import kv_reference as ref
from tests.test_gpu_paged_attention import make_cache

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def attention(q, k, v, n, *, causal, window, sinks, scale):
    """As kv_reference.attention, from one table of what sees what."""
    length, group = k.shape[0], q.shape[1] // k.shape[1]
    j, p = torch.arange(length)[None], (length - n + torch.arange(n))[:, None]
    seen = (j > p - window) | (j < sinks) if window else torch.ones((n, length), dtype=torch.bool)
    if causal:
        seen = seen & (j <= p)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    w_abs, p_abs, dots = torch.zeros_like(q), torch.zeros_like(q), 0.0
    for h in range(q.shape[1]):
        kk, vv = k[:, h // group], v[:, h // group]
        s = torch.where(seen, (q[:, h] @ kk.T) * scale, -math.inf)
        if length and n:
            dots = max(dots, float((q[:, h].abs() @ kk.abs().T).max()) * scale)
        lse[:, h] = torch.logsumexp(s, 1)
        w = torch.where(seen, torch.exp(s - lse[:, h:h + 1]), 0.0)
        out[:, h], w_abs[:, h], p_abs[:, h] = w @ vv, w @ vv.abs(), seen.double() @ vv.abs()
    return out, lse, w_abs, p_abs, dots


def check(case, *, seed=0, max_new=None, stream=None):
    dtype, dim, q_heads, kv_heads, page, seqs, causal, window, sinks = case
    gen = torch.Generator().manual_seed(seed)
    lens = [n for _, n in seqs]
    cache, pool, table = make_cache(gen, lens, dtype=dtype, dim=dim, kv_heads=kv_heads, page=page)
    clean, entries = pool.clone(), table.clone()
    for r, (n, length) in enumerate(seqs):  # what lies between the first tokens and the window
        first = max(0, length - n - window + 1) if window else 0
        hidden = [j for j in range(first) if j >= sinks]
        for j in hidden:
            pool[table[r, j // page], :, :, :, j % page] = math.nan
        for i in {j // page for j in hidden}:
            if i * page >= sinks and (i + 1) * page <= first:
                entries[r, i] = [-1, 10**6, -(2**31)][i % 3]
    cache.pool.copy_(pool)
    cache.table.copy_(entries)
    cu = [0]
    for n, _ in seqs:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], q_heads, dim), generator=gen).to(dtype)
    scale = 1.0 / math.sqrt(dim)
    got, lse = api.paged_attention(q.cuda(), cache, 0, torch.tensor(cu, dtype=torch.int32).cuda(), causal=causal, window=window, sinks=sinks,
                                   max_new=max_new, return_lse=True, stream=stream)
    assert cache.status(stream=stream) == 0
    u = ref.UNIT[dtype]
    for s, (n, length) in enumerate(seqs):
        k, v = ref.row_tokens(clean, table, 0, s, length)
        want, want_lse, w_abs, p_abs, dots = attention(q[cu[s]:cu[s + 1]].double(), k, v, n, causal=causal, window=window, sinks=sinks,
                                                       scale=scale)
        score_err = dim * 2.0**-24 * dots
        tol = u * want.abs() + (u + 2 * score_err + 2.0**-20) * w_abs + (2.0**-24 if dtype == F16 else 0.0) * (1 + p_abs)
        have, have_lse = got[cu[s]:cu[s + 1]].cpu().double(), lse[cu[s]:cu[s + 1]].cpu().double()
        assert ((have - want).abs() <= 2 * tol).all(), (s, float(((have - want).abs() / (tol + 1e-30)).max()))
        empty = want_lse == -math.inf
        assert (have_lse[empty] == -math.inf).all() and (have[empty] == 0).all()
        assert ((have_lse - want_lse)[~empty].abs() <= 2 * (score_err + 2.0**-20 * (1 + want_lse[~empty].abs()))).all()
    return got, lse


CASES = {
    # dtype, head_dim, q_heads, kv_heads, page, [(new, length)], causal, window, sinks
    "one_token": (BF16, 128, 4, 1, 16, [(1, 3000)], True, 100, 4),
    "lengths_around_the_window": (F16, 64, 4, 2, 16, [(1, n) for n in (1, 2, 3, 4, 5, 99, 100, 101, 103, 104, 105, 128, 129, 257)], True, 100, 4),
    "tile_edges": (BF16, 64, 2, 1, 16, [(1, n) for n in (255, 256, 257, 383, 384, 385, 511, 512, 513, 640)], True, 128, 128),
    "sinks_past_a_tile": (F16, 128, 2, 2, 32, [(1, 2000), (3, 700), (2, 300), (1, 130)], True, 60, 129),
    "sinks_end_in_the_windows_tile": (BF16, 64, 4, 2, 16, [(1, 260), (4, 250), (1, 200)], True, 50, 135),
    "sinks_and_window_touch": (F16, 64, 2, 1, 16, [(1, 104), (1, 105), (1, 103), (5, 108)], True, 100, 4),
    "more_sinks_than_tokens": (BF16, 64, 2, 1, 16, [(1, 40), (7, 300), (1, 900)], True, 10, 500),
    "window_of_one": (F16, 128, 4, 4, 16, [(1, 500), (5, 321), (2, 2)], True, 1, 1),
    "draft_block": (BF16, 128, 32, 8, 16, [(7, 300), (7, 7), (7, 5025), (7, 64), (7, 140)], False, 128, 20),
    "chunk": (F16, 128, 4, 1, 128, [(150, 1411), (40, 40), (33, 700)], True, 90, 70),
    "chunk_longer_than_the_window": (BF16, 64, 2, 1, 64, [(515, 1515)], True, 33, 5),
    "prompt": (F16, 64, 3, 1, 32, [(700, 700), (1, 1), (300, 301)], True, 64, 16),
    "odd_group": (BF16, 64, 7, 1, 32, [(37, 2290), (100, 100)], True, 200, 9),
    "pages_longer_than_a_tile": (F16, 64, 2, 2, 256, [(3, 3000), (1, 511), (1, 514)], True, 300, 260),
    "chunk_longer_than_its_row": (BF16, 64, 4, 4, 16, [(2, 0), (3, 1), (5, 3), (1, 17)], True, 2, 1),
    "split": (BF16, 128, 4, 1, 64, [(1, 30000)], True, 20000, 700),
    "split_chunk": (F16, 128, 4, 1, 64, [(32, 12000), (1, 300)], True, 9000, 300),
    "split_pairs": (BF16, 64, 3, 1, 128, [(49, 12720)] * 2, True, 8000, 2000),
    "many": (F16, 64, 2, 1, 16, [(1 + i % 3, 1 + 137 * i % 1211) for i in range(70)], True, 77, 5),
    "whole_items": (BF16, 64, 8, 2, 16, [(130, 1130), (0, 9), (257, 300), (1, 1), (64, 2900)], True, 50, 3),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name):
    check(CASES[name], seed=len(name))


@pytest.mark.parametrize("max_new", [1, 7, 4000])
def test_the_hint_only_costs_time(max_new):
    check((F16, 64, 4, 2, 16, [(70, 900), (1, 400), (130, 131)], True, 100, 20), max_new=max_new, seed=7)


def test_on_another_stream():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    check(CASES["draft_block"], stream=side)


def test_without_sinks_or_window_nothing_changes():
    gen = torch.Generator().manual_seed(3)
    cache, _, _ = make_cache(gen, [900, 33], dtype=BF16, dim=128, kv_heads=2, page=16, poison=False)
    q = torch.randn((12, 8, 128), generator=gen).to(BF16).cuda()
    cu = torch.tensor([0, 7, 12], dtype=torch.int32).cuda()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    whole = api.paged_attention(q, cache, 0, cu)
    assert same(api.paged_attention(q, cache, 0, cu, sinks=9), whole)               # no window: all is visible
    assert same(api.paged_attention(q, cache, 0, cu, window=2**31 - 1, sinks=2**31 - 1), whole)
    assert same(api.paged_attention(q, cache, 0, cu, window=900, sinks=4), whole)    # a window of all
    assert same(api.paged_attention(q, cache, 0, cu, window=50, sinks=2**31 - 1), whole) or torch.allclose(
        api.paged_attention(q, cache, 0, cu, window=50, sinks=2**31 - 1).float(), whole.float(), atol=0.02)
    assert not same(api.paged_attention(q, cache, 0, cu, window=50, sinks=4), api.paged_attention(q, cache, 0, cu, window=50))
    with pytest.raises(api.DsparkError):
        api.paged_attention(q, cache, 0, cu, window=50, sinks=-1)


def test_in_a_graph_with_a_growing_row():
    gen = torch.Generator().manual_seed(4)
    cache, pool, table = make_cache(gen, [600], dtype=BF16, dim=64, kv_heads=1, page=16, poison=False)
    q = torch.randn((1, 2, 64), generator=gen).to(BF16).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    api.paged_attention(q, cache, 0, cu, window=64, sinks=4, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_attention(q, cache, 0, cu, window=64, sinks=4, out=out)
    for length in (600, 1, 68, 69, 129, 300):
        cache.length.fill_(length)
        graph.replay()
        torch.cuda.synchronize()
        k, v = ref.row_tokens(pool, table, 0, 0, length)
        want, _, w_abs, _, _ = attention(q.cpu().double(), k, v, 1, causal=True, window=64, sinks=4, scale=0.125)
        assert ((out.cpu().double() - want).abs() <= 2 * (2.0**-8 * (want.abs() + w_abs) + 1e-4 * w_abs)).all()
