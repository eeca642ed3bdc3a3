"""Rotary positions, alone and into the cache, against a 64-bit reference.

Tolerance: the result is rounded once (unit roundoff u of its type); the angle is exact to 2^-32 of a turn, its
fp32 form to 2^-25 of a half turn, sine and cosine to a few units of 2^-24 and the two products and the sum to
2^-24 each: 2^-20 of |a| + |b| covers them."""
import math

import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def plain_freqs(rotary_dim, base=10000.0):
    return [base ** (-2.0 * j / rotary_dim) / (2.0 * math.pi) for j in range(rotary_dim // 2)]


def tolerance(x, want, dtype, amplitude):
    size = x.double().abs().amax(-1, keepdim=True) * 2 * amplitude
    return ref.UNIT[dtype] * want.abs() + 2.0**-20 * size + (2.0**-24 if dtype == F16 else 0.0)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("tokens,heads,dim,rotary_dim", [(1, 1, 128, 128), (3, 40, 128, 64), (67, 7, 64, 16),
                                                         (1000, 2, 80, 48), (33, 5, 512, 512), (5, 130, 16, 16)])
def test_against_64_bits(tokens, heads, dim, rotary_dim, dtype, layout, backward):
    gen = torch.Generator().manual_seed(tokens + dim)
    x = torch.randn((tokens, heads, dim), generator=gen).to(dtype)
    pos = torch.randint(-5000, 2_000_000, (tokens,), generator=gen, dtype=torch.int32)
    pos[0] = 0 if tokens == 1 else 2**31 - 1
    table = api.RotaryTable(api.rotary_frequencies(rotary_dim), layout=layout, amplitude=1.25)
    got = api.rotary(x.cuda(), pos.cuda(), table, backward=backward)
    want = ref.rotary(x.double(), pos, plain_freqs(rotary_dim), layout=layout, amplitude=1.25, backward=backward)
    # the reference's own angle loses 2^-53 of the whole turns: 2^31 / 2 pi * 2^-53 of a turn is far below
    err = (got.cpu().double() - want).abs()
    assert (err <= 2 * tolerance(x, want, dtype, 1.25)).all(), float(err.max())
    assert torch.equal(got[..., rotary_dim:].cpu(), x[..., rotary_dim:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_in_place(layout):
    gen = torch.Generator().manual_seed(3)
    fused = torch.randn((50, 12, 64), generator=gen).to(BF16).cuda()
    pos = torch.arange(50, dtype=torch.int32).cuda()
    table = api.RotaryTable(api.rotary_frequencies(32), layout=layout)
    want = api.rotary(fused[:, 2:9].contiguous(), pos, table)
    rest = fused.clone()
    out = api.rotary(fused[:, 2:9], pos, table, out=fused[:, 2:9])
    assert torch.equal(out, want) and torch.equal(fused[:, :2], rest[:, :2]) and torch.equal(fused[:, 9:], rest[:, 9:])
    head_major = rest.permute(1, 0, 2).contiguous().permute(1, 0, 2)  # tokens next to each other
    assert torch.equal(api.rotary(head_major[:, 2:9], pos, table), want)


def test_gradient_against_differences():
    # y is linear in x, so (L(x + h e) - L(x - h e)) / 2h is the gradient of L = <w, y> up to roundings
    gen = torch.Generator().manual_seed(4)
    x, w = (torch.randn((4, 2, 32), generator=gen, dtype=torch.float64).float().cuda() for _ in range(2))
    pos = torch.tensor([0, 1, 777, 100000], dtype=torch.int32).cuda()
    for layout in ("half", "interleaved"):
        table = api.RotaryTable(api.rotary_frequencies(16), layout=layout, amplitude=0.75)
        grad = api.rotary(w, pos, table, backward=True)
        h = 0.5
        for i in range(0, 4):
            for e in range(32):
                step = torch.zeros_like(x)
                step[i, 1, e] = h
                up, down = api.rotary(x + step, pos, table), api.rotary(x - step, pos, table)
                diff = ((up.double() - down.double()) * w.double()).sum() / (2 * h)
                # each of the two products' terms is off by at most 2^-20 of values below 8
                assert abs(float(diff - grad[i, 1, e].double())) <= 2.0**-20 * 8 * 4


def test_backward_undoes_forward():
    gen = torch.Generator().manual_seed(5)
    x = torch.randn((200, 3, 128), generator=gen).cuda()
    pos = torch.randint(0, 1 << 20, (200,), generator=gen, dtype=torch.int32).cuda()
    table = api.RotaryTable(api.rotary_frequencies(128), layout="interleaved")
    back = api.rotary(api.rotary(x, pos, table), pos, table, backward=True)
    assert ((back - x).abs() <= 2.0**-19 * 8).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,rotary_dim,layout,page", [(128, 128, "half", 16), (64, 16, "interleaved", 64),
                                                        (128, 32, "half", 256)])
def test_append(dtype, dim, rotary_dim, layout, page):
    gen = torch.Generator().manual_seed(dim + page)
    seqs = [(1, 1), (5, 40), (0, 12), (20, 20), (3, 259)]  # new, length with them
    rows = [3, 0, 4, 1, 2]
    heads, kv, layers, layer = 6, 2, 3, 1
    cache = api.PagedCache.empty(200, 5, 20, layers=layers, kv_heads=kv, page_size=page, head_dim=dim, dtype=dtype)
    cache.pool.copy_(torch.randn(cache.pool.shape, generator=gen).to(dtype))
    r = torch.tensor(rows, dtype=torch.int32).cuda()
    cache.extend(r, torch.tensor([n for _, n in seqs], dtype=torch.int32).cuda())
    before = cache.pool.cpu().clone()
    total = sum(n for n, _ in seqs)
    cu = [0]
    for n, _ in seqs:
        cu.append(cu[-1] + n)
    fused = torch.randn((total + 2, heads + 2 * kv, dim), generator=gen).to(dtype)
    dev = fused.cuda()
    table = api.RotaryTable(api.rotary_frequencies(rotary_dim, 500000.0), layout=layout, amplitude=1.5)
    q, k, v = dev[:, :heads], dev[:, heads : heads + kv], dev[:, heads + kv :]
    out = torch.full((total + 2, heads, dim), 9.0, dtype=dtype, device="cuda")
    api.rotary_append(q, k, v, cache, layer, torch.tensor(cu, dtype=torch.int32).cuda(), table, rows=r, out=out)
    assert cache.status() == 0
    assert (out[total:] == 9.0).all()  # tokens of no sequence
    pos = torch.tensor([length - n + i for n, length in seqs for i in range(n)])
    freqs = plain_freqs(rotary_dim, 500000.0)
    x = fused[:total].double()
    want_q = ref.rotary(x[:, :heads], pos, freqs, layout=layout, amplitude=1.5)
    want_k = ref.rotary(x[:, heads : heads + kv], pos, freqs, layout=layout, amplitude=1.5)
    assert ((out[:total].cpu().double() - want_q).abs() <= 2 * tolerance(x[:, :heads], want_q, dtype, 1.5)).all()
    after, books, t = cache.pool.cpu(), cache.table.cpu(), 0
    for (n, length), row in zip(seqs, rows):
        for i in range(n):
            p = length - n + i
            at = (books[row, p // page], layer)
            slot = p % page
            assert ((after[at][0, :, slot].double() - want_k[t]).abs()
                    <= 2 * tolerance(x[t, heads : heads + kv], want_k[t], dtype, 1.5)).all()
            assert torch.equal(after[at][1, :, slot], fused[t, heads + kv :])
            before[at][0, :, slot], before[at][1, :, slot] = after[at][0, :, slot], after[at][1, :, slot]
            t += 1
    assert torch.equal(before, after)  # nothing else was written


def test_append_with_positions_of_its_own_and_places_that_do_not_exist():
    cache = api.PagedCache.empty(8, 2, 4, layers=1, kv_heads=1, page_size=16, head_dim=64, dtype=BF16)
    cache.pool.zero_()
    cache.extend(torch.tensor([0], dtype=torch.int32).cuda(), torch.tensor([2], dtype=torch.int32).cuda())
    gen = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn((3, 1, 64), generator=gen).to(BF16).cuda() for _ in range(3))
    table = api.RotaryTable(api.rotary_frequencies(64))
    pos = torch.tensor([70, 71, 72], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 3], dtype=torch.int32).cuda()
    out = api.rotary_append(q, k, v, cache, 0, cu, table, positions=pos)
    assert cache.status() == api.DSPARK_ERR_INDEX  # three tokens for a row of two: the first has no place
    assert torch.equal(out, api.rotary(q, pos, table))
    page = int(cache.table[0, 0])
    turned = api.rotary(k, pos, table)
    assert torch.equal(cache.pool[page, 0, 0, 0, :2], turned[1:, 0]) and torch.equal(cache.pool[page, 0, 1, 0, :2], v[1:, 0])
    assert (cache.pool[page, 0, :, :, 2:] == 0).all() and int((cache.pool != 0).any(-1).sum()) == 4


def test_refusals():
    table = api.RotaryTable(api.rotary_frequencies(64))
    x = torch.zeros((4, 2, 64), dtype=BF16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")

    def refused(status, *a, **kw):
        with pytest.raises(api.DsparkError) as e:
            api.rotary(*a, **kw)
        assert e.value.status == status

    refused(api.DSPARK_ERR_UNSUPPORTED, x[..., :48], pos, table)
    refused(api.DSPARK_ERR_UNSUPPORTED, x, pos, api.RotaryTable(api.rotary_frequencies(24)))
    refused(api.DSPARK_ERR_UNSUPPORTED, torch.zeros((4, 2, 72), dtype=BF16, device="cuda"), pos, table)
    wide = torch.zeros((4, 2, 68), dtype=BF16, device="cuda")
    refused(api.DSPARK_ERR_INVALID, wide[..., 4:], pos, table)
    for bad in (x.double(), x[0], x.cpu(), x.transpose(1, 2)):
        with pytest.raises(ValueError):
            api.rotary(bad, pos, table)
    with pytest.raises(ValueError):
        api.rotary(x, pos[:3], table)
    with pytest.raises(ValueError):
        api.rotary(x, pos.long(), table)
    with pytest.raises(ValueError):
        api.rotary(x, pos, table, out=x[:2])
    with pytest.raises(ValueError):
        api.RotaryTable(table.turns, layout="quarter")
    assert api.rotary(x[:0], pos[:0], table).shape == (0, 2, 64)
    cache = api.PagedCache.empty(8, 2, 4, layers=1, kv_heads=1, page_size=16, head_dim=64, dtype=BF16)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        api.rotary_append(x, x, x, cache, 0, cu, table)
    with pytest.raises(api.DsparkError):
        api.rotary_append(x, x[:, :1], x[:, 1:], cache, 1, cu, table)
