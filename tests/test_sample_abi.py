"""The sampling calls without a GPU: arguments are refused before the device is touched, on the C side and in the binding."""
import math
import os
import subprocess

import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests.test_kv_devices import Stream, World, ints, on

INVALID, UNSUPPORTED = api.DSPARK_ERR_INVALID, api.DSPARK_ERR_UNSUPPORTED
FAKE, ODD = 0x10000, 0x10001  # never dereferenced


def sample(lib, logits=FAKE, uniforms=FAKE, ids=FAKE, probs=0, stride=100, probs_stride=100, dtype=2, rows=3, vocab=100, t=0, p=0, m=0, k=0, temperature=1.0,
           top_p=1.0, min_p=0.0, top_k=0):
    return lib.dspark_sample(api._SAMPLE_ARGS.pack(logits, uniforms, ids, probs, stride, probs_stride, dtype, rows, vocab, t, p, m, k, temperature, top_p,
                                                   min_p, top_k), None)


def verify(lib, logits=FAKE, uniforms=FAKE, cu=FAKE, drafts=FAKE, probs=0, ids=FAKE, accepted=FAKE, stride=100, probs_stride=100, dtype=2, vocab=100, seqs=2,
           n=5, t=0, p=0, m=0, k=0, temperature=1.0, top_p=1.0, min_p=0.0, top_k=0):
    return lib.dspark_verify_drafts(api._VERIFY_ARGS.pack(logits, uniforms, cu, drafts, probs, ids, accepted, stride, probs_stride, dtype, vocab, seqs, n, t, p,
                                                          m, k, temperature, top_p, min_p, top_k), None)


BAD = [(dict(logits=0), INVALID), (dict(uniforms=0), INVALID), (dict(ids=0), INVALID), (dict(logits=ODD), INVALID), (dict(uniforms=0x10002), INVALID),
       (dict(ids=0x10004), INVALID), (dict(probs=0x10002), INVALID), (dict(vocab=0), INVALID), (dict(vocab=-1), INVALID), (dict(vocab=(1 << 19) + 1), UNSUPPORTED),
       (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(stride=-1), INVALID), (dict(temperature=-0.1), INVALID), (dict(temperature=math.nan), INVALID),
       (dict(top_p=-0.1), INVALID), (dict(top_p=1.5), INVALID), (dict(top_p=math.nan), INVALID), (dict(min_p=-0.1), INVALID), (dict(min_p=1.1), INVALID),
       (dict(min_p=math.nan), INVALID), (dict(top_k=-1), INVALID), (dict(t=0x10002), INVALID), (dict(k=0x10002), INVALID)]


@pytest.mark.parametrize("change,status", BAD)
def test_what_both_calls_refuse(dspark_lib, change, status):
    assert sample(dspark_lib, **change) == status and dspark_lib.dspark_last_error().decode()
    assert verify(dspark_lib, **change) == status and dspark_lib.dspark_last_error().decode()


def test_what_each_refuses(dspark_lib):
    lib = dspark_lib
    assert lib.dspark_sample(None, None) == INVALID and lib.dspark_verify_drafts(None, None) == INVALID
    assert sample(lib, rows=-1) == INVALID and sample(lib, probs=FAKE, probs_stride=99) == INVALID
    assert sample(lib, rows=1 << 28) == UNSUPPORTED
    assert sample(lib, rows=0, logits=0, uniforms=0, ids=0) == 0
    for kw in (dict(cu=0), dict(drafts=0), dict(accepted=0), dict(cu=0x10002), dict(drafts=0x10004), dict(accepted=0x10002), dict(seqs=-1), dict(n=-1),
               dict(probs=FAKE, probs_stride=-1)):
        assert verify(lib, **kw) == INVALID, kw
    assert verify(lib, seqs=1 << 30, n=(1 << 30) + 5) == UNSUPPORTED and verify(lib, seqs=1 << 28) == UNSUPPORTED
    assert verify(lib, seqs=0, n=0, logits=0, uniforms=0, cu=0, drafts=0, ids=0, accepted=0) == 0


def test_argument_structs_have_the_sizes_of_the_header(dspark_lib, tmp_path):
    names = {"dspark_sample_args": api._SAMPLE_ARGS.size, "dspark_verify_args": api._VERIFY_ARGS.size}
    src = tmp_path / "sizes.c"
    src.write_text('#include "dspark.h"\n' + "".join(f"_Static_assert(sizeof({n}) == {s}, \"{n}\");\n" for n, s in names.items()))
    subprocess.run(["gcc", "-fsyntax-only", "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include"), str(src)],
                   check=True)


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def floats(index, *shape):
    return on(index, *shape, dtype=torch.float32)


def test_calls_go_to_the_tensors_gpu(world):
    x, u = floats(1, 4, 50), floats(1, 4)
    api.sample(x, u, out=ints(1, 4, dtype=torch.int64))
    api.verify_drafts(x, ints(1, 2, dtype=torch.int64), ints(1, 3), floats(1, 4, 2), out=ints(1, 4, dtype=torch.int64), accepted=ints(1, 2))
    assert [c[0] for c in world.calls] == ["dspark_sample", "dspark_verify_drafts"]
    assert all(c[1] == 1 for c in world.calls) and world.current == 0
    with pytest.raises(ValueError):
        api.sample(x, u, out=ints(1, 4, dtype=torch.int64), stream=Stream(0))


def test_tensors_that_are_refused(world):
    x, u, out = floats(0, 4, 50), floats(0, 4), ints(0, 4, dtype=torch.int64)
    good = dict(out=out)
    for bad in (x.double(), x.T, x[0], torch.zeros(4, 50), ints(0, 4, 50)):
        with pytest.raises(ValueError):
            api.sample(bad, u, **good)
    for bad in (floats(1, 4), floats(0, 3), u.double(), floats(0, 8)[::2]):
        with pytest.raises(ValueError):
            api.sample(x, bad, **good)
    for kw in (dict(out=ints(0, 4)), dict(out=ints(0, 5, dtype=torch.int64)), dict(temperature=floats(0, 3)), dict(temperature=floats(1, 4)),
               dict(top_k=floats(0, 4)), dict(top_p=ints(0, 4)), dict(min_p=floats(0, 5)), dict(probs=floats(0, 4, 49)), dict(probs=floats(0, 3, 50)),
               dict(probs=on(0, 4, 50, dtype=torch.float16)), dict(probs=floats(0, 50, 4).T)):
        with pytest.raises(ValueError):
            api.sample(x, u, **{**good, **kw})
    drafts, cu, u2 = ints(0, 2, dtype=torch.int64), ints(0, 3), floats(0, 4, 2)
    good = dict(out=out, accepted=ints(0, 2))
    for args in ((x, ints(0, 3, dtype=torch.int64), cu, u2), (x, drafts, ints(0, 4), u2), (x, drafts, cu, u), (x, ints(0, 2), cu, u2), (x, drafts, cu.long(), u2),
                 (x, ints(1, 2, dtype=torch.int64), cu, u2)):
        with pytest.raises(ValueError):
            api.verify_drafts(*args, **good)
    for kw in (dict(accepted=ints(0, 3)), dict(draft_probs=floats(0, 3, 50)), dict(draft_probs=floats(0, 2, 49)), dict(draft_probs=on(0, 2, 50)),
               dict(temperature=floats(0, 4))):
        with pytest.raises(ValueError):
            api.verify_drafts(x, drafts, cu, u2, **{**good, **kw})
    assert world.calls == []
