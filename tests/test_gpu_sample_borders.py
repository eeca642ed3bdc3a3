"""Drawing and judging where a row's number falls on tokens of next to no weight, where a filter ends among equal logits, and where
uniform numbers lie outside 0..1.  Ids have to be equal to the 64-bit reference's; the cases are made so that no border between two tokens is
nearer to a number than the weights' error allows."""
import math

import numpy as np
import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests import sample_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
INF, NAN = math.inf, math.nan


def at_offset(x, offset):
    """x on the GPU, its rows `offset` elements behind a 16-byte boundary and next to NaN."""
    rows, vocab = x.shape
    per = 16 // x.element_size()
    wide = torch.full((rows, -(-(vocab + offset) // per) * per + per), NAN, dtype=x.dtype, device="cuda")
    wide[:, offset:offset + vocab] = x
    return wide[:, offset:offset + vocab]


def offsets(dtype):
    return range(16 // torch.tensor([], dtype=TYPES[dtype]).element_size())


# ---- numbers that fall on tokens of less than 2^-44 of the heaviest ----

@pytest.mark.parametrize("hidden", [-INF, NAN])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_light_tokens_behind_a_masked_one(dtype, hidden):
    """The first 32 bytes hold a masked token and ones of exp(-30.8), 0.74 of 2^-44 of the heaviest: none of them is a unit of the sums, all
    together are some.  u = 0 draws the first that is a token.

    With u so that u z = 2, the sum up to what is drawn, itself included, is above 2, as sums are never rounded up; the sum before it is at most 2
    and one for each vector that ended before it, as a vector's sum is cut to whole units.  A vector has 16 bytes of a slice at least."""
    t = TYPES[dtype]
    for vocab in (40, 700, 4099, 20000):
        x = torch.full((3, vocab), -30.8)
        x[:, 18:] = -INF
        x[:, vocab // 2:vocab // 2 + 8] = 0.0
        x[0, 0] = x[2, 0] = hidden
        x[2, 1] = hidden
        x = x.to(t)
        light = np.exp(x[:, :18].double().numpy()) * 2.0**44
        light = np.where(np.isnan(light), 0.0, light)
        for offset in offsets(dtype):
            for u in (0.0, -1.0, NAN, 2.0**-46):
                ids = api.sample(at_offset(x, offset), torch.full((3,), u, device="cuda")).tolist()
                if u > 0:
                    for r, i in enumerate(ids):
                        assert i < 18 and light[r, i] > 0 and light[r, :i + 1].sum() > 2, (vocab, offset, r, i)
                        assert light[r, :i].sum() <= 2 + -(-i // (16 // x.element_size())), (vocab, offset, r, i)
                else:
                    assert ids == [1, 0, 2], (vocab, offset, u)
                    assert ids == [ref.pick(ref.distribution(row), 0.0) for row in x.double().numpy()]


@pytest.mark.parametrize("dtype", list(TYPES))
def test_light_tokens_that_a_filter_leaves(dtype):
    """The same where 1200 tokens weigh one each and the settings leave the first 1300 (top_k), or all that are no lighter (min_p): too many to
    be listed."""
    t = TYPES[dtype]
    vocab = 4001
    x = torch.full((2, vocab), -INF)
    x[:, 1:301] = -30.8
    x[:, 2000:3200] = 0.0
    x[1, 0] = NAN
    x = x.to(t)
    for kw in (dict(top_k=1300), dict(min_p=1e-14), dict(top_k=1300, min_p=1e-14)):
        want = [ref.distribution(r, **kw) for r in x.double().numpy()]
        for offset in offsets(dtype):
            ids, p = api.sample(at_offset(x, offset), torch.zeros(2, device="cuda"), return_probs=True, **kw)
            assert ids.tolist() == [1, 1] == [ref.pick(w, 0.0) for w in want]
            assert ((p.cpu().numpy() > 0) == (want[0] > 0)).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rests_of_light_tokens_behind_a_masked_one(dtype):
    """A refused draft whose rest has, in its first 32 bytes, only tokens of about 0.7 of 2^-62 each."""
    t = TYPES[dtype]
    vocab = 5000
    x = torch.full((2, vocab), -INF)
    x[:, 1:16] = -41.25  # exp(-41.25) / 8 = 0.69 of 2^-62
    x[:, 3000:3008] = 0.0
    x = x.to(t)
    q = torch.zeros((1, vocab))
    q[0, 3005] = 1.0
    u = torch.tensor([[0.9, 0.0], [0.5, 0.5]])
    p = ref.distribution(x[0].double().numpy())
    want, taken = ref.verify([p, p], [3005], u.numpy(), q.numpy())
    assert want == [1, -1] and taken == 0
    for offset in offsets(dtype):
        ids, n = api.verify_drafts(at_offset(x, offset), torch.tensor([3005], device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), u.cuda(),
                                   draft_probs=q.cuda())
        assert ids.tolist() == want and n.tolist() == [0], offset


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rests_that_are_rounding_alone(dtype):
    """The drafts' distribution is the target's rounded to 32 bits, but for what the refused draft has too much: what is left of most tokens is the
    rounding of q.  Whatever a number falls on has to be a token of the row, and one whose p is not below q by more than p's error: 2^-22 of
    the fast exponential, 2^-24 for each of four roundings and for q's own, and |ln w| 2^-24 of the difference of logits, |ln w| < 22 here: 2^-19."""
    t = TYPES[dtype]
    gen = torch.Generator().manual_seed(31)
    seqs, vocab = 96, 3001
    x = torch.randn((2 * seqs, vocab), generator=gen) * 2
    keep = torch.rand((2 * seqs, vocab), generator=gen) < 0.2  # one or two tokens of 32 bytes
    x = torch.where(keep, x, -INF).to(t)
    p = np.stack([ref.distribution(r) for r in x[::2].double().numpy()])
    q = torch.from_numpy(p).float()
    drafts = q.argmax(1)
    q[torch.arange(seqs), drafts] = 1.0
    cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    for u1 in (0.0, 1e-9, 3e-9, 0.3, 0.999999):
        u = torch.tensor([[0.9999, u1]]).expand(2 * seqs, 2).contiguous()
        for offset in (0, 1):
            ids, n = api.verify_drafts(at_offset(x, offset), drafts.cuda(), cu, u.cuda(), draft_probs=q.cuda())
            assert n.tolist() == [0] * seqs
            got = ids.cpu()[::2].numpy()
            at = np.arange(seqs)
            assert ((got >= 0) & (got < vocab)).all() and (p[at, got] > 0).all()
            assert (p[at, got] >= q.double().numpy()[at, got] * (1 - 2.0**-19)).all()


# ---- filters that end among equal logits ----

@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("settings", [dict(top_k=600), dict(top_p=0.5), dict(top_k=900, top_p=0.7), dict(top_k=1001), dict()])
def test_min_p_drops_the_logit_that_another_filter_ended_on(settings, dtype, per_row):
    """One token of logit 0 and 1000 of -1, of which top_k or top_p leaves some hundred: too many to be listed.  min_p is exp(-1) rounded up, by 2.5e-8
    of itself where a weight is off by 2^-27 = 7.5e-9 at most, so that one token is left."""
    vocab, min_p = 2500, float(np.float32(math.exp(-1)))
    assert min_p > math.exp(-1) * (1 + 2.0**-26)
    x = torch.full((2, vocab), -INF)
    x[:, 700:1700] = -1.0
    x[:, 1234] = 0.0
    x = x.to(TYPES[dtype]).cuda()
    kw = dict(settings, min_p=min_p)
    if per_row:
        kw = {n: torch.full((2,), v, dtype=torch.int32 if n == "top_k" else torch.float32, device="cuda") for n, v in kw.items()}
    u = torch.tensor([0.0, 0.999], device="cuda")
    ids, p = api.sample(x, u, return_probs=True, **kw)
    assert ids.tolist() == [1234, 1234]
    assert (p[:, 1234] == 1).all() and (p != 0).sum() == 2
    # no draft of the others is accepted
    one = {n: v[:1] if per_row else v for n, v in kw.items()}
    for draft, want in ((700, [1234, -1]), (1234, [1234, 1234])):
        ids, n = api.verify_drafts(x, torch.tensor([draft], device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                   torch.tensor([[0.0, 0.7], [0.5, 0.2]], device="cuda"), **one)
        assert ids.tolist() == want and n.tolist() == [int(draft == 1234)]


# ---- uniform numbers outside 0..1 ----

@pytest.mark.parametrize("settings", [dict(), dict(top_k=5), dict(top_p=0.9), dict(temperature=0.0)])
def test_judging_by_numbers_outside_their_range(settings):
    """u0 below 0 or NaN is 0, 1 and above just below 1: a draft that the target never takes is not accepted, one that it always takes is."""
    vocab, k = 1000, 7
    u = torch.rand((k + 1, 2), generator=torch.Generator().manual_seed(3))
    cu = torch.tensor([0, k], dtype=torch.int32, device="cuda")
    x = torch.randn((k + 1, vocab), generator=torch.Generator().manual_seed(4))
    x[:, 17] = -INF
    best = x.argmax(1)
    for q in (None, torch.full((k, vocab), 1.0 / vocab, device="cuda")):
        for u0 in (-0.5, -INF, NAN, 0.0):
            u[:, 0] = u0
            ids, n = api.verify_drafts(x.cuda(), torch.full((k,), 17, device="cuda"), cu, u.cuda(), draft_probs=q, **settings)
            assert n.tolist() == [0] and ids[0] != 17 and ids[0] >= 0, (u0, q is None)
            ids, n = api.verify_drafts(x.cuda(), best[:k].cuda(), cu, u.cuda(), draft_probs=q, **settings)
            assert n.tolist() == [k] and ids[:k].tolist() == best[:k].tolist(), (u0, q is None)
    one = torch.full((k + 1, vocab), -INF)
    one[:, 33] = 2.0
    for u0 in (1.0, 1.5, INF):
        u[:, 0] = u0
        ids, n = api.verify_drafts(one.cuda(), torch.full((k,), 33, device="cuda"), cu, u.cuda(), **settings)
        assert n.tolist() == [k] and (ids == 33).all(), u0


# ---- what is dropped has no probability at all ----

@pytest.mark.parametrize("dtype", list(TYPES))
def test_dropped_tokens_have_a_probability_of_zero(dtype):
    """Exactly 0, whatever stands in for them on the way; and what is left sums to 1 (each value is off by 2^-21 of itself at most, and by
    |ln w| 2^-24, which is largest where w is least: w |ln w| < 0.4)."""
    t = TYPES[dtype]
    gen = torch.Generator().manual_seed(41)
    far = float(torch.finfo(t).max) / 4
    settings = [(1.0, 0, 1.0, 0.0), (0.7, 40, 1.0, 0.0), (1.3, 700, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (8.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.01), (2.0, 900, 0.8, 0.001),
                (0.0, 0, 1.0, 0.0), (1e-3, 0, 1.0, 0.0), (1e4, 0, 0.6, 0.0)]
    for vocab in (300, 5003):
        for shift, spread in ((0.0, 3.0), (-1000.0, 3.0), (1000.0, 30.0), (0.0, far), (-far, 1.0)):
            x = (torch.randn((len(settings), vocab), generator=gen).clamp(-3, 3) * spread + shift).to(t)
            x[:, 3::7] = -INF
            x[:, 5::11] = NAN
            columns = [torch.tensor(c) for c in zip(*settings)]
            kw = dict(temperature=columns[0].float().cuda(), top_k=columns[1].int().cuda(), top_p=columns[2].float().cuda(), min_p=columns[3].float().cuda())
            _, p = api.sample(x.cuda(), torch.full((len(settings),), 0.5, device="cuda"), return_probs=True, **kw)
            p = p.cpu().double().numpy()
            for r, (temperature, k, top_p, m) in enumerate(settings):
                host = x[r].double().numpy()
                f = lambda v: float(np.float32(v))  # noqa: E731
                want = ref.distribution(host, f(temperature), k, 1.0, f(m))  # top_p's end may lie between two tokens: what the others leave
                assert (p[r][~(host > -INF)] == 0).all() and (p[r][want == 0] == 0).all(), (vocab, shift, spread, settings[r])
                kept = np.flatnonzero(p[r])
                if top_p < 1:  # the first ones of the order
                    order = np.lexsort((np.arange(vocab), -np.where(host > -INF, host, -INF)))
                    assert set(kept) == set(order[:len(kept)])
                assert abs(p[r].sum() - 1) < 2.0**-20, (vocab, shift, spread, settings[r])
