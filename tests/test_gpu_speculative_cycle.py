"""The example's cycle: the cache it leaves holds what appending the kept tokens alone would have left."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_cycle.py")


def test_cycle_runs_and_leaves_a_sound_cache():
    spec = importlib.util.spec_from_file_location("speculative_cycle", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    cache = example.main(["--cycles", "3", "--requests", "5"])
    lengths, table = cache.length.tolist(), cache.table.cpu()
    assert lengths[5:] == [0] * 5 and (table[5:] == -1).all()
    held = torch.zeros(cache.refs.numel(), dtype=torch.int32)
    for r, n in enumerate(lengths[:5]):
        pages = -(-n // 16)
        assert 20 + 13 * r + 3 <= n <= 20 + 13 * r + 21  # one to seven tokens a cycle
        assert (table[r, :pages] >= 0).all() and (table[r, pages:] == -1).all()
        held.index_add_(0, table[r, :pages].long(), torch.ones(pages, dtype=torch.int32))
    assert torch.equal(held, cache.refs.cpu())
