"""Which GPU the key-value calls run on, and that they refuse tensors spread over several: on the CPU, with tensors that only
say where they are and a library that only notes its calls."""
import contextlib

import pytest
import torch

from dspark_draft_sampling_gb300 import api


class Tensor(torch.Tensor):
    """A CPU tensor that says it is on the GPU `index`."""
    index = 0

    def get_device(self):
        return self.index

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)


def on(index, *shape, dtype=torch.float16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Tensor)
    t.index = index
    return t


def ints(index, *shape, dtype=torch.int32):
    return on(index, *shape, dtype=dtype)


class Stream:
    def __init__(self, index):
        self.device_index, self.device, self.cuda_stream = index, torch.device("cuda", index), 77


class World:
    """Two GPUs, of which one is current, and the calls made."""

    def __init__(self, monkeypatch):
        self.current, self.calls = 0, []

        @contextlib.contextmanager
        def device(index):
            before, self.current = self.current, torch.device("cuda", index).index if isinstance(index, int) else index.index
            yield
            self.current = before

        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index)
        monkeypatch.setattr(api, "load_library", lambda: self)

    def __getattr__(self, name):
        if not name.startswith("dspark_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, self.current, args[-1]))
            return 0

        return call


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def cache(index, **change):
    t = dict(pool=on(index, 8, 1, 2, 2, 16, 64), table=ints(index, 4, 2), length=ints(index, 4), refs=ints(index, 8))
    t.update(change)
    return api.PagedCache(t["pool"], t["table"], t["length"], t["refs"], workspace=change.get("workspace", on(index, 4096)))


def calls(index, c, stream=None, **change):
    """Every call of the key-value side, by name, with one tensor or more elsewhere."""
    t = dict(rows=ints(index, 2), other=ints(index, 2), kept=ints(index, 2, 3), q=on(index, 4, 4, 64), k=on(index, 4, 2, 64),
             v=on(index, 4, 2, 64), out=on(index, 4, 4, 64), cu=ints(index, 3), pos=ints(index, 4),
             lse=on(index, 4, 4, dtype=torch.float32), turns=ints(index, 16, dtype=torch.int64))
    t.update(change)
    table = api.RotaryTable(t["turns"])
    return {
        "extend": lambda: c.extend(t["rows"], t["other"], stream=stream),
        "fork": lambda: c.fork(t["rows"], t["other"], stream=stream),
        "compact": lambda: c.compact(t["rows"], t["other"], t["kept"], t["other"], stream=stream),
        "free": lambda: c.free(t["rows"], stream=stream),
        "copy_pages": lambda: c.copy_pages(t["rows"], t["other"], stream=stream),
        "status": lambda: c.status(stream=stream),
        "rotary": lambda: api.rotary(t["q"], t["pos"], table, out=t["out"], stream=stream),
        "rotary_append": lambda: api.rotary_append(t["q"], t["k"], t["v"], c, 0, t["cu"], table, rows=t["rows"], positions=t["pos"],
                                                   out=t["out"], stream=stream),
        "paged_attention": lambda: api.paged_attention(t["q"], c, 0, t["cu"], rows=t["rows"], out=t["out"], lse=t["lse"], stream=stream),
    }


NAMES = ["extend", "fork", "compact", "free", "copy_pages", "status", "rotary", "rotary_append", "paged_attention"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_the_gpu_of_their_tensors(world, name, index):
    c = cache(index)
    for stream, raw in ((None, 1000 + index), (Stream(index), 77)):
        world.calls.clear()
        calls(index, c, stream)[name]()
        assert [call[1:] for call in world.calls] == [(index, raw)]
        assert world.current == 0


USES = [("rows", "extend"), ("other", "extend"), ("rows", "fork"), ("other", "fork"), ("rows", "compact"), ("other", "compact"),
        ("kept", "compact"), ("rows", "free"), ("rows", "copy_pages"), ("other", "copy_pages")]
USES += [(t, "rotary") for t in ("q", "pos", "out", "turns")]
USES += [(t, "rotary_append") for t in ("q", "k", "v", "cu", "rows", "pos", "out", "turns")]
USES += [(t, "paged_attention") for t in ("q", "cu", "rows", "out", "lse")]
SHAPES = dict(rows=(2,), other=(2,), kept=(2, 3), q=(4, 4, 64), k=(4, 2, 64), v=(4, 2, 64), out=(4, 4, 64), cu=(3,), pos=(4,), lse=(4, 4),
              turns=(16,))
TYPES = dict(q=torch.float16, k=torch.float16, v=torch.float16, out=torch.float16, lse=torch.float32, turns=torch.int64)


@pytest.mark.parametrize("tensor,name", USES)
def test_a_tensor_on_another_gpu_is_refused(world, tensor, name):
    c = cache(0)
    run = calls(0, c, **{tensor: on(1, *SHAPES[tensor], dtype=TYPES.get(tensor, torch.int32))})[name]
    with pytest.raises(ValueError):
        run()
    assert not world.calls


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_gpu_is_refused(world, name):
    with pytest.raises(ValueError):
        calls(0, cache(0), Stream(1))[name]()
    assert not world.calls


@pytest.mark.parametrize("name,t", [("table", ints(1, 4, 2)), ("length", ints(1, 4)), ("refs", ints(1, 8)), ("workspace", on(1, 4096))])
def test_a_cache_over_several_gpus_is_refused(world, name, t):
    with pytest.raises(ValueError):
        cache(0, **{name: t})
