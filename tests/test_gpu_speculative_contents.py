"""The example's cycle leaves in its cache what appending the kept tokens alone leaves: nothing of rejected drafts, nothing at
another position.

Tolerance: both caches hold the same projections, rounded to fp16 (unit roundoff 2^-11) from 32-bit sums of 1024 terms whose
order may differ with the rows beside them: an fp16 step and 2^-16 of |w||x| (below 8 here) on each of a pair's two elements, and
after the rotation another rounding; angles and their sines are the same in both."""
import importlib.util
import os

import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_cycle.py")


def test_cycle_leaves_what_appending_the_kept_tokens_leaves():
    spec = importlib.util.spec_from_file_location("speculative_cycle", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    n = 5
    cache, layer, prompts, accepted = example.run(n, 3)
    kept = [torch.cat([prompts[r]] + [chunk[r, :keep[r]] for chunk, keep in accepted]) for r in range(n)]
    lens = [len(k) for k in kept]
    assert cache.length[:n].tolist() == lens and any(int(keep.max()) < 7 for _, keep in accepted)

    fresh = api.PagedCache.empty(n * 16, n, 16, layers=1, kv_heads=example.KV_HEADS, page_size=16, head_dim=example.DIM,
                                 dtype=torch.float16)
    rows, cu = example.ints(range(n)), example.ints([sum(lens[:i]) for i in range(n + 1)])
    fresh.extend(rows, example.ints(lens))
    layer.forward(torch.cat(kept), fresh, cu, rows, max(lens), causal=True)
    assert fresh.status() == 0

    def tolerance(x):  # of a pair's two elements, twice rounded; the other half of the head holds its partner
        half = x.shape[-1] // 2
        pair = x.abs() + x.abs().roll(half, -1)
        return 2 * (2 * 2.0**-11 * pair + 2 * 8 * 2.0**-16)

    for r in range(n):
        got = ref.row_tokens(cache.pool.cpu(), cache.table.cpu(), 0, r, lens[r])
        want = ref.row_tokens(fresh.pool.cpu(), fresh.table.cpu(), 0, r, lens[r])
        for a, b in zip(got, want):
            assert ((a - b).abs() <= tolerance(b)).all(), (r, float((a - b).abs().max()))
        # a neighbouring position's key would be far outside
        assert ((got[0][1:] - want[0][:-1]).abs() > tolerance(want[0][:-1])).any(-1).all()
