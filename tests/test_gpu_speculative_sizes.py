"""The example's cycle with more requests and longer lives than its defaults: its cache is as large as they need."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_cycle.py")


@pytest.mark.parametrize("requests,cycles", [(41, 2), (2, 75), (1, 1)])
def test_cycle_of_other_sizes(requests, cycles):
    spec = importlib.util.spec_from_file_location("speculative_cycle", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    cache = example.main(["--cycles", str(cycles), "--requests", str(requests)])
    for r, n in enumerate(cache.length.tolist()[:requests]):
        assert 20 + 13 * r + cycles <= n <= 20 + 13 * r + 7 * cycles
