"""The cache operators' C entries without a GPU: arguments are refused before the device is touched."""
import ctypes
import math
import os

import pytest

from dspark_draft_sampling_gb300 import api

INVALID, UNSUPPORTED = api.DSPARK_ERR_INVALID, api.DSPARK_ERR_UNSUPPORTED
FAKE, ODD = 0x10000, 0x10004  # never dereferenced


def cache(**kw):
    a = dict(pool=FAKE, table=FAKE, length=FAKE, refs=FAKE, workspace=FAKE, workspace_bytes=1 << 30, dtype=1, num_pages=64,
             layers=2, kv_heads=2, page_size=16, head_dim=128, max_seqs=4, max_pages=8)
    a.update(kw)
    return ctypes.byref(api.CacheStruct(**a))


BAD_CACHES = [(dict(pool=None), INVALID), (dict(table=None), INVALID), (dict(length=None), INVALID), (dict(refs=None), INVALID),
              (dict(workspace=None), INVALID), (dict(pool=ODD), INVALID), (dict(refs=ODD), INVALID), (dict(workspace=ODD), INVALID),
              (dict(workspace_bytes=256), INVALID), (dict(num_pages=0), INVALID), (dict(layers=0), INVALID),
              (dict(kv_heads=-1), INVALID), (dict(max_seqs=0), INVALID), (dict(max_pages=0), INVALID),
              (dict(page_size=0), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
              (dict(page_size=512), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
              (dict(num_pages=1 << 24), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED)]


def attend(lib, c, layer=0, q=FAKE, qs=(512, 128), tokens=3, heads=4, cu=FAKE, seqs=1, max_new=3, window=0, out=FAKE,
           os=(512, 128), lse=0, scale=1.0):
    return lib.dspark_paged_attention(c, api._ATTENTION_ARGS.pack(q, out, lse, 0, cu, *qs, *os, layer, tokens, heads, seqs, max_new, 1,
                                                                  window, scale), None)


def append(lib, c, layer=0, q=FAKE, k=FAKE, v=FAKE, out=FAKE, stride=512, tokens=3, heads=4, cu=FAKE, seqs=1, turns=FAKE, dim=128,
           layout=0):
    return lib.dspark_rotary_append(c, api._APPEND_ARGS.pack(q, k, v, out, 0, cu, 0, turns, *(stride, 128) * 4, layer, tokens, heads, seqs,
                                                             dim, layout, 1.0), None)


def turn(lib, x=FAKE, y=FAKE, stride=512, dtype=1, tokens=3, heads=4, head_dim=128, pos=FAKE, turns=FAKE, dim=128, layout=0):
    return lib.dspark_rotary(api._ROTARY_ARGS.pack(x, y, pos, turns, stride, 128, stride, 128, dtype, tokens, heads, head_dim, dim, layout,
                                                   0, 1.0), None)


def test_argument_structs_have_the_sizes_of_the_header(dspark_lib, tmp_path):
    import subprocess
    names = {"dspark_rotary_args": api._ROTARY_ARGS.size, "dspark_append_args": api._APPEND_ARGS.size,
             "dspark_attention_args": api._ATTENTION_ARGS.size, "dspark_cache": ctypes.sizeof(api.CacheStruct)}
    src = tmp_path / "sizes.c"
    src.write_text('#include "dspark.h"\n' + "".join(f"_Static_assert(sizeof({n}) == {s}, \"{n}\");\n" for n, s in names.items()))
    subprocess.run(["gcc", "-fsyntax-only", "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include"),
                    str(src)], check=True)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_caches_that_are_refused(dspark_lib, change, status):
    lib, c = dspark_lib, cache(**change)
    assert lib.dspark_cache_extend(c, FAKE, FAKE, 1, None) == status
    assert lib.dspark_cache_status(c, None) == status
    assert attend(lib, c) == status and append(lib, c) == status
    assert lib.dspark_last_error().decode()


def test_page_operations_refuse(dspark_lib):
    lib, c = dspark_lib, cache()
    assert lib.dspark_cache_extend(None, FAKE, FAKE, 1, None) == INVALID
    assert lib.dspark_cache_extend(c, None, FAKE, 1, None) == INVALID
    assert lib.dspark_cache_extend(c, FAKE, None, 1, None) == INVALID
    assert lib.dspark_cache_extend(c, FAKE, FAKE, -1, None) == INVALID
    assert lib.dspark_cache_extend(c, FAKE, FAKE, 5, None) == INVALID  # more rows than the table has
    assert lib.dspark_cache_extend(cache(max_seqs=5000), FAKE, FAKE, 1025, None) == UNSUPPORTED
    assert lib.dspark_cache_fork(c, FAKE, None, 1, None) == INVALID
    assert lib.dspark_cache_free(c, None, 1, None) == INVALID
    assert lib.dspark_cache_compact(c, FAKE, FAKE, FAKE, -1, FAKE, 1, None) == INVALID
    assert lib.dspark_cache_compact(c, FAKE, FAKE, None, 3, FAKE, 1, None) == INVALID
    assert lib.dspark_cache_compact(c, FAKE, FAKE, FAKE, 3, None, 1, None) == INVALID
    assert lib.dspark_cache_compact(c, FAKE, None, None, 0, None, 1, None) == INVALID
    assert lib.dspark_cache_copy_pages(c, FAKE, None, 1, None) == INVALID
    assert lib.dspark_cache_copy_pages(c, FAKE, FAKE, -1, None) == INVALID
    for name in ("extend", "fork", "copy_pages"):
        assert getattr(lib, "dspark_cache_" + name)(c, None, None, 0, None) == 0
    assert lib.dspark_cache_free(c, None, 0, None) == 0
    assert lib.dspark_cache_compact(c, None, None, None, 0, None, 0, None) == 0


def test_workspace_bytes(dspark_lib):
    size = dspark_lib.dspark_cache_workspace_bytes
    assert size(cache(pool=None, workspace=None)) >= 1024
    assert size(cache(max_seqs=1024, max_pages=100000)) > size(cache())
    assert size(cache(page_size=17)) == 0 and size(None) == 0


def test_attention_refuses(dspark_lib):
    lib, c = dspark_lib, cache()
    for kw in (dict(layer=2), dict(layer=-1), dict(q=0), dict(out=0), dict(cu=0), dict(q=ODD), dict(out=ODD), dict(lse=0x10002),
               dict(tokens=-1), dict(heads=0), dict(heads=3), dict(seqs=-1), dict(max_new=-1), dict(window=-1), dict(qs=(516, 128)),
               dict(os=(512, 129)), dict(qs=(-512, 128)), dict(qs=(0, 128)), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan)):
        assert attend(lib, c, **kw) == INVALID, kw
    assert attend(lib, c, heads=258) == UNSUPPORTED
    assert attend(lib, c, seqs=4097) == UNSUPPORTED
    assert attend(lib, c, tokens=0) == 0 and attend(lib, c, seqs=0) == 0
    assert lib.dspark_paged_attention(c, None, None) == INVALID and lib.dspark_rotary_append(c, None, None) == INVALID
    assert lib.dspark_rotary(None, None) == INVALID


def test_rotary_refuses(dspark_lib):
    lib, c = dspark_lib, cache()
    for kw in (dict(turns=0), dict(turns=ODD), dict(layout=2), dict(stride=516), dict(tokens=-1)):
        assert append(lib, c, **kw) == INVALID, kw
        assert turn(lib, **kw) == INVALID, kw
    for kw in (dict(dim=120), dict(dim=8), dict(dim=144), dict(dim=0)):
        assert append(lib, c, **kw) == UNSUPPORTED and turn(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(layer=2), dict(k=0), dict(v=ODD), dict(q=0), dict(out=0), dict(cu=0), dict(seqs=-1)):
        assert append(lib, c, **kw) == INVALID, kw
    assert append(lib, c, seqs=4097) == UNSUPPORTED
    for kw in (dict(x=0), dict(y=ODD), dict(pos=0), dict(dtype=3), dict(heads=-1)):
        assert turn(lib, **kw) == INVALID, kw
    assert turn(lib, head_dim=136) == UNSUPPORTED and turn(lib, head_dim=528) == UNSUPPORTED
    assert turn(lib, tokens=0) == 0 and turn(lib, heads=0) == 0 and append(lib, c, tokens=0) == 0


def test_frequencies():
    turn_ = 2.0**64
    plain = api.rotary_frequencies(64, 10000.0)
    for j, f in enumerate(plain):
        want = 10000.0 ** (-2 * j / 64) / (2 * math.pi)
        assert abs((f % 2**64) / turn_ - want) <= 2.0**-52
    linear = api.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert all(abs(a % 2**64 * 4.0 / (b % 2**64) - 1) < 1e-12 for a, b in zip(linear, plain))
    raised = api.rotary_frequencies(64, scaling="base", factor=4.0)
    assert raised[0] == plain[0] and abs(raised[-1] * 4.0 / plain[-1] - 1) < 1e-12
    parts = api.rotary_frequencies(64, scaling="by_parts", factor=8.0, original=4096)
    turns = [10000.0 ** (-2 * j / 64) / (2 * math.pi) * 4096 for j in range(32)]
    for t, a, b in zip(turns, parts, plain):
        if t >= 32:
            assert a == b
        elif t <= 1:
            assert abs(a * 8.0 / b - 1) < 1e-12
        else:
            assert b / 8 < a < b
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=4, base=0.0), dict(rotary_dim=4, scaling="x"),
                dict(rotary_dim=4, scaling="linear", factor=0.5), dict(rotary_dim=4, scaling="by_parts", factor=2.0)):
        with pytest.raises(ValueError):
            api.rotary_frequencies(**bad)
