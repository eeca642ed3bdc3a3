"""The cache's page operations against books kept as lists: tables, lengths, counts and moved tokens are equal."""
import random

import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests.kv_reference import Books

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Pair:
    """A cache and its books, driven together and compared after every call."""

    def __init__(self, pages, rows, wide, *, page=16, layers=2, heads=3, dim=64, dtype=torch.bfloat16, seed=0):
        self.cache = api.PagedCache.empty(pages, rows, wide, layers=layers, kv_heads=heads, page_size=page, head_dim=dim,
                                          dtype=dtype)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.cache.pool.copy_(torch.randn(self.cache.pool.shape, generator=gen, device="cuda"))
        self.books = Books(pages, wide, page, rows)

    def call(self, name, *args):
        before = self.cache.pool.clone()
        self.books.moves = []
        done = getattr(self.books, name)(*args)
        if name == "compact":
            rows, start, kept = args
            wide = max(map(len, kept)) + 1
            full = [list(k) + [-7] * (wide - len(k)) for k in kept]  # what lies behind n_kept is not looked at
            self.cache.compact(ints(rows), ints(start), ints(full), ints([len(k) for k in kept]))
        else:
            getattr(self.cache, name)(*map(ints, args))
        assert self.cache.status() == (0 if done is not False else api.DSPARK_ERR_CAPACITY)
        assert torch.equal(self.cache.table.cpu(), self.books.table())
        assert self.cache.length.tolist() == list(self.books.length.values())
        assert self.cache.refs.tolist() == self.books.refs()
        want = self.books.moved(before) if done is not False else before
        assert torch.equal(self.cache.pool.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("page,dim,dtype", [(16, 64, torch.bfloat16), (64, 128, torch.float16)])
def test_a_life(page, dim, dtype):
    p = Pair(60, 8, 9, page=page, dim=dim, dtype=dtype)
    p.call("extend", [0, 3, 5], [page * 3, page * 2 + 5, 1])
    p.call("extend", [3, 0, 1], [page - 5, 0, 7])
    p.call("fork", [3, 3, 5], [4, 6, 2])
    p.call("extend", [4, 6], [2, page + 1])
    p.call("fork", [4, 6, 3], [6, 3, 4])  # a cycle of rows
    p.call("fork", [0, 1], [0, 2])        # a row onto itself stays
    p.call("compact", [6], [3], [[5, 6, 9, page, 2 * page]])  # in a shared page
    p.call("compact", [4, 0], [0, page], [[1, 2, 3], []])
    p.call("free", [3, 7, 0])
    p.call("extend", [7], [page * 9])
    p.call("free", [1, 2, 4, 5, 6, 7])
    assert not p.cache.refs.any()


def test_random_life():
    r = random.Random(1)
    p = Pair(300, 24, 12, page=16, layers=1, heads=1)
    for _ in range(60):
        rows = r.sample(range(24), r.randint(1, 24))
        op = r.choice(["extend", "extend", "fork", "compact", "compact", "free"])
        if op == "extend":
            p.call("extend", rows, [r.choice([0, 1, 3, 16, 40]) for _ in rows])
        elif op == "fork":
            p.call("fork", [r.randrange(24) for _ in rows], rows)
        elif op == "free":
            p.call("free", rows[:3])
        else:
            start = [r.randint(0, p.books.length[x]) for x in rows]
            kept = [sorted(r.sample(range(s, p.books.length[x]), r.randint(0, p.books.length[x] - s)))
                    for x, s in zip(rows, start)]
            p.call("compact", rows, start, kept)


def test_capacity_is_all_or_nothing():
    p = Pair(4, 4, 3)
    p.call("extend", [0, 1], [40, 16])
    p.call("extend", [1, 2], [16, 1])   # five pages of four
    p.call("fork", [0, 1], [2, 3])      # the copy of a last page does not fit
    p.call("extend", [1], [33])         # a row of at most three pages
    p.call("free", [1])
    p.call("fork", [0], [2])
    p.call("compact", [2], [3], [[4, 20]])  # the first page is shared, and none is free
    p.call("free", [0, 2])


def test_many_pages_and_rows():
    # more pages than one pass of the scan takes, and more rows than a warp has lanes
    p = Pair(40000, 1024, 60, layers=1, heads=1)
    p.call("extend", list(range(1024)), [(7 * i) % 500 for i in range(1024)])
    p.call("free", list(range(0, 1024, 3)))
    p.call("extend", list(range(0, 1024, 3))[::-1], [(11 * i) % 900 for i in range(342)])
    p.call("fork", [i ^ 1 for i in range(1024)], list(range(1024)))


@pytest.mark.parametrize("page,dim", [(16, 128), (128, 64)])
def test_long_compaction(page, dim):
    r = random.Random(2)
    p = Pair(700 * 16 // page, 4, 250 * 16 // page, page=page, dim=dim, layers=1, heads=2)
    p.call("extend", [0, 1, 2], [3900, 2047, 130])
    p.call("compact", [1, 0], [4, 4], [list(range(36, 2047)), sorted(r.sample(range(4, 3900), 1777))])
    p.call("fork", [0], [3])
    p.call("compact", [3, 0], [100, 0], [sorted(r.sample(range(100, 1781), 900)), list(range(5, 1781))])


def test_many_runs():
    # more runs of layers and heads than there are SMs, and so many forks that several share a block
    r = random.Random(4)
    p = Pair(420, 330, 7, page=64, dim=128, layers=6, heads=8)
    p.call("extend", [0, 1, 2, 3], [400, 129, 64, 333])
    p.call("compact", [0, 3, 1], [4, 0, 10],
           [list(range(40, 400)), sorted(r.sample(range(333), 200)), list(range(64, 129))])
    p.call("fork", [r.choice([0, 0, 0, 1, 2, 3]) for _ in range(7)] + [i // 37 % 4 for i in range(7, 326)], list(range(4, 330)))


def test_cut_off_without_a_list():
    p = Pair(20, 3, 8)
    p.call("extend", [0, 1], [50, 33])
    p.books.compact([0, 1], [17, 0], [[], []])
    p.cache.compact(ints([0, 1]), ints([17, 0]))
    assert p.cache.status() == 0
    assert torch.equal(p.cache.table.cpu(), p.books.table()) and p.cache.length.tolist() == [17, 0, 0]
    assert p.cache.refs.tolist() == p.books.refs()


def test_copy_pages():
    p = Pair(30, 2, 4, layers=3, heads=5, dim=128)
    want = p.cache.pool.clone()
    want[[4, 9, 2]] = want[[7, 7, 29]]
    p.cache.copy_pages(ints([7, 7, 29]), ints([4, 9, 2]))
    assert p.cache.status() == 0 and torch.equal(p.cache.pool, want)
    p.cache.copy_pages(ints([1, 30, 3]), ints([8, 5, -1]))
    want[8] = want[1]
    assert p.cache.status() == api.DSPARK_ERR_INDEX and torch.equal(p.cache.pool, want)


def test_bad_indices_change_nothing():
    p = Pair(20, 3, 4)
    p.call("extend", [0, 1], [40, 20])
    books = [t.clone() for t in (p.cache.table, p.cache.length, p.cache.refs, p.cache.pool)]
    c = p.cache
    kept = ints([[5, 7, 7], [1, 2, 3]])
    for call in (lambda: c.extend(ints([0, 3]), ints([1, 1])), lambda: c.extend(ints([0, 1]), ints([1, -1])),
                 lambda: c.fork(ints([0, -1]), ints([1, 2])), lambda: c.fork(ints([0]), ints([3])),
                 lambda: c.free(ints([0, 4])),
                 lambda: c.compact(ints([0, 1]), ints([5, 1]), kept, ints([3, 2])),   # not ascending
                 lambda: c.compact(ints([0, 1]), ints([6, 1]), kept, ints([1, 1])),   # before start
                 lambda: c.compact(ints([0, 1]), ints([0, 1]), ints([[39, 40], [1, 2]]), ints([2, 1])),
                 lambda: c.compact(ints([0, 1]), ints([41, 1]), kept, ints([0, 1])),
                 lambda: c.compact(ints([0, 1]), ints([5, 1]), kept, ints([4, 1]))):
        call()
        assert c.status() == api.DSPARK_ERR_INDEX
        for t, was in zip((c.table, c.length, c.refs, c.pool), books):
            assert torch.equal(t, was)
    assert c.status() == 0


def test_refusals():
    c = api.PagedCache.empty(8, 2, 4, layers=1, kv_heads=1, page_size=16, head_dim=64)
    with pytest.raises(ValueError):
        c.extend(ints([0]), ints([1, 2]))
    with pytest.raises(ValueError):
        c.extend(ints([0]).long(), ints([1]))
    with pytest.raises(ValueError):
        c.compact(ints([0]), ints([0]), ints([1]), ints([0]))
    with pytest.raises(api.DsparkError) as e:
        c.free(ints([0, 1, 0]))
    assert e.value.status == api.DSPARK_ERR_INVALID
    for sizes in (dict(page_size=24, head_dim=64), dict(page_size=8, head_dim=64), dict(page_size=512, head_dim=64),
                  dict(page_size=16, head_dim=80)):
        with pytest.raises(api.DsparkError) as e:
            api.PagedCache.empty(8, 2, 4, layers=1, kv_heads=1, **sizes)
        assert e.value.status == api.DSPARK_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        api.PagedCache(c.pool, c.table, c.length[:1], c.refs)
    with pytest.raises(ValueError):
        api.PagedCache(c.pool.float(), c.table, c.length, c.refs)
    with pytest.raises(api.DsparkError):
        api.PagedCache(c.pool, c.table, c.length, c.refs, workspace=c.workspace[:512]).free(ints([0]))
    c.free(ints([])), c.extend(ints([]), ints([]))
    assert c.status() == 0
