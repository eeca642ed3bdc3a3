"""paged_attention's number of first tokens on its way into the library: on the CPU, with a library that only notes its calls."""
import pytest

from dspark_draft_sampling_gb300 import api
from tests.test_kv_devices import World, cache, ints, on


class Noting(World):
    def __getattr__(self, name):
        if not name.startswith("dspark_"):
            raise AttributeError(name)
        c_types = api.SIGNATURES[name][1]

        def call(*args):  # numbers as C has them
            self.calls.append((name, *[t(v).value for t, v in zip(c_types, args) if isinstance(v, int)]))
            return 0

        return call


@pytest.mark.parametrize("sinks,passed", [(0, None), (4, 4), (2**31 - 1, 2**31 - 1), (2**31, 2**31 - 1), (2**32, 2**31 - 1), (2**32 + 4, 2**31 - 1),
                                          (2**70, 2**31 - 1), (-1, -1), (-(2**32), -1), (-(2**32) + 7, -1)])
def test_numbers_beyond_32_bits_are_all_tokens_or_refused(monkeypatch, sinks, passed):
    world = Noting(monkeypatch)
    c = cache(0)
    api.paged_attention(on(0, 3, 2, 64), c, 0, ints(0, 2), window=8, sinks=sinks, out=on(0, 3, 2, 64))
    (name, *numbers), = world.calls
    if passed is None:
        assert name == "dspark_paged_attention"
    else:
        assert name == "dspark_paged_attention_sinks" and numbers[0] == passed


def test_a_number_that_is_not_whole_is_refused(dspark_lib):
    args = api._ATTENTION_ARGS.pack(*[0] * 16, 1.0)
    with pytest.raises(Exception):
        dspark_lib.dspark_paged_attention_sinks(None, args, 4.5, None)
