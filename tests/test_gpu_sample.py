"""Drawing tokens and judging drafts against the 64-bit reference, at the sizes, types and settings where they can go wrong.

Ids have to be equal.  A uniform number closer than 1e-7 of the row's mass to a border between two tokens says nothing (weights are off by
2^-27, or 2^-27 of the heaviest one's, and the reference's own sums by 1e-16): such numbers are moved before the first run, in `away`.
The distribution is rounded to fp32: the light weights' fast exponential is off by 2^-22, their product, the sum's and its reciprocal's
rounding and the last product by 2^-24 each, so less than 2^-21 of a value together; and a light weight's difference of logits d is rounded
to 32 bits, |d| 2^-24, so its weight exp(d / T) by 2^-24 of |d / T| = |ln w| of itself."""
import math

import numpy as np
import pytest
import torch

from dspark_draft_sampling_gb300 import api
from tests import sample_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CLOSE = 1e-7


def away(p, u):
    """u, or the next number that is not on a border of p."""
    u = np.float32(u)
    while p.any() and ref.margin(p, float(u)) < CLOSE:
        u = np.float32(u + 3e-6) if u < 0.9 else np.float32(u - 0.17)
    return u


def clear(l, top_p, temperature=1.0, top_k=0):
    """Whether the nucleus' end is clear: no token's mass before it is within 1e-8 of top_p."""
    p = np.sort(ref.distribution(l, temperature, top_k))[::-1]
    before = np.concatenate(([0.0], np.cumsum(p)[:-1]))
    before = before[p > 0]
    return np.abs(before - np.float64(np.float32(top_p))).min() > 1e-8


def logits_of(gen, rows, vocab, dtype, spread=2.0):
    x = torch.randn((rows, vocab), generator=gen) * spread
    n = min(40, vocab // 2)
    if n:
        x.scatter_add_(1, torch.randint(0, vocab, (rows, n), generator=gen), torch.rand((rows, n), generator=gen) * 8)
    return x.to(dtype)


def f32(v):
    return float(np.float32(v))


def check(logits, settings, gen, *, probs=False, strided=0, scalar=False, stream=None):
    """settings: a list of (temperature, top_k, top_p, min_p) for the rows, or one for all (scalar)."""
    rows, vocab = logits.shape
    host = logits.double().numpy()
    per_row = [settings] * rows if scalar else settings
    want = [ref.distribution(host[r], f32(t), k, f32(p), f32(m)) for r, (t, k, p, m) in enumerate(per_row)]
    u = torch.rand(rows, generator=gen).numpy()
    u = np.array([away(p, x) for p, x in zip(want, u)], dtype=np.float32)
    x = logits.cuda()
    if strided:  # rows that are not next to each other, and start at any element
        wide = torch.full((rows, vocab + strided), math.nan, dtype=logits.dtype, device="cuda")
        wide[:, 1:1 + vocab] = x
        x = wide[:, 1:1 + vocab]
    if scalar:
        kw = dict(zip(("temperature", "top_k", "top_p", "min_p"), settings))
    else:
        t, k, p, m = zip(*settings)
        kw = dict(temperature=torch.tensor(t, dtype=torch.float32).cuda(), top_k=torch.tensor(k, dtype=torch.int32).cuda(),
                  top_p=torch.tensor(p, dtype=torch.float32).cuda(), min_p=torch.tensor(m, dtype=torch.float32).cuda())
    got = api.sample(x, torch.from_numpy(u).cuda(), return_probs=probs, **kw)
    ids, have = got if probs else (got, None)
    ids = ids.cpu().tolist()
    for r in range(rows):
        assert ids[r] == ref.pick(want[r], float(u[r])), (r, per_row[r], u[r], ids[r], ref.pick(want[r], float(u[r])))
        if probs:
            h = have[r].cpu().double().numpy()
            assert ((h > 0) == (want[r] > 1e-13)).all() or (np.abs(h - want[r]) <= 1e-12)[(h > 0) != (want[r] > 1e-13)].all(), r
            log = np.abs(np.log(np.where(want[r] > 0, want[r], 1.0) / max(want[r].max(), 1e-300))) * (want[r] > 0)
            assert (np.abs(h - want[r]) <= want[r] * (2.0**-21 + 2.0**-24 * log) + 1e-13).all(), (r, per_row[r])
    return ids


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 0, 1.0, 0.0), (1.0, 5, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.1), (0.9, 40, 0.95, 0.05),
            (0.0, 0, 1.0, 0.0), (1.0, 1, 0.5, 0.5), (5.0, 700, 0.99, 0.0), (0.2, 0, 0.3, 0.0), (3.0, 0, 0.997, 0.0), (30.0, 0, 0.5, 0.0)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 64, 500, 1001, 4096, 32000, 50257])
def test_every_setting_in_one_batch(vocab, dtype):
    gen = torch.Generator().manual_seed(vocab)
    x = logits_of(gen, len(SETTINGS), vocab, TYPES[dtype])
    keep = [i for i, (t, k, p, m) in enumerate(SETTINGS) if t == 0 or p == 1 or clear(x[i].double().numpy(), p, t, k)]
    assert len(keep) >= len(SETTINGS) - 1
    check(x[keep], [SETTINGS[i] for i in keep], gen, probs=True, strided=3)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("setting", [SETTINGS[0], SETTINGS[5], SETTINGS[3], (1.0, 0, 0.999, 0.0), (1.0, 3000, 1.0, 0.0), (1.5, 5000, 0.9, 0.001)])
@pytest.mark.parametrize("rows,vocab", [(1, 151936), (3, 248319)])
def test_large_vocabularies(rows, vocab, setting, dtype):
    gen = torch.Generator().manual_seed(rows)
    check(logits_of(gen, rows, vocab, TYPES[dtype], 2.5), setting, gen, probs=True, scalar=True)


def test_the_largest_vocabulary():
    gen = torch.Generator().manual_seed(3)
    check(logits_of(gen, 2, 1 << 19, torch.float32, 3.0), [(1.0, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.0)], gen, probs=True)


@pytest.mark.parametrize("rows", [1, 2, 9, 38, 39, 77, 152, 153, 700])
def test_a_row_draws_the_same_alone_and_among_others(rows):
    gen = torch.Generator().manual_seed(rows)
    x = logits_of(gen, rows, 3001, torch.float32).cuda()
    u = torch.rand(rows, generator=gen).cuda()
    for kw in (dict(), dict(top_k=30), dict(top_p=0.9), dict(temperature=2.0, top_p=0.99, min_p=0.001)):
        ids, probs = api.sample(x, u, return_probs=True, **kw)
        for r in {0, rows // 2, rows - 1}:
            one, p = api.sample(x[r:r + 1], u[r:r + 1], return_probs=True, **kw)
            assert one[0] == ids[r] and torch.equal(p[0], probs[r])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_masks(dtype):
    gen = torch.Generator().manual_seed(5)
    t, vocab = TYPES[dtype], 2003
    x = logits_of(gen, 14, vocab, t)
    low = torch.finfo(t).min
    inf = math.inf
    x[0] = -inf                       # nothing left
    x[1] = math.nan
    x[2] = -inf
    x[2, vocab - 1] = -3.0            # one token
    x[3] = low                        # all of the type's lowest value: tokens like any others
    x[4, :2000] = low                 # lowest beside ordinary ones
    x[5, 7::2] = -inf
    x[6, ::3] = math.nan              # NaN among ordinary ones
    x[7, 40] = inf                    # one +infinity
    x[8, [3, 900, 2002]] = inf        # three
    x[9] = -inf
    x[9, [5, 1200]] = low             # two tokens of the lowest value among masked ones
    x[10] = torch.finfo(t).max        # all of the highest
    x[11] = -inf
    x[11, :3] = torch.tensor([torch.finfo(t).max, low, 0.0])
    x[12] = 0.0
    x[12, ::2] = -0.0                 # equal, whatever their sign
    x[13, 100:] = -inf
    u = torch.linspace(0.05, 0.95, 14)
    for setting in ((1.0, 0, 1.0, 0.0), (1.0, 3, 1.0, 0.0), (1.0, 0, 0.77, 0.0), (1.0, 0, 1.0, 0.2), (0.0, 0, 1.0, 0.0), (1e4, 50, 0.93, 0.01)):
        check(x, setting, gen, probs=True, scalar=True)
    ids = api.sample(x.cuda(), u.cuda()).cpu().tolist()
    assert ids[:3] == [-1, -1, vocab - 1] and ids[7] == 40
    assert api.sample(x.cuda(), u.cuda(), temperature=0.0).cpu()[12] == 0


@pytest.mark.parametrize("dtype", list(TYPES))
def test_many_infinities_and_highest_values(dtype):
    """More equal largest logits than one block lists, beyond where differences are finite."""
    gen = torch.Generator().manual_seed(6)
    t, vocab = TYPES[dtype], 6007
    x = logits_of(gen, 3, vocab, t)
    x[0, 1::3] = math.inf
    x[1, ::2] = torch.finfo(t).max
    x[2, ::5] = math.inf
    x[2, 1::5] = torch.finfo(t).min
    for setting in ((1.0, 0, 0.7071, 0.0), (0.5, 900, 1.0, 0.0), (1.0, 700, 0.3333, 0.5), (1.0, 0, 1.0, 0.5), (0.0, 0, 1.0, 0.0)):
        check(x, setting, gen, probs=True, scalar=True)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_ties(dtype):
    """Few distinct logits: equal ones stay by index, wherever the last one of them lies."""
    gen = torch.Generator().manual_seed(8)
    for vocab in (513, 9000, 40001):
        x = (torch.randint(0, 5, (6, vocab), generator=gen).float() * 0.5).to(TYPES[dtype])
        x[0] = 1.25
        p = 0.6180339
        settings = [(1.0, 300, 1.0, 0.0), (1.0, 3, 1.0, 0.0), (0.8, vocab // 3 + 1, 1.0, 0.0), (1.1, 0, p, 0.0), (0.5, vocab // 2, p, 0.1), (1.0, 0, 0.11111, 0.0)]
        assert all(clear(x[r].double().numpy(), s[2], s[0], s[1]) for r, s in enumerate(settings) if s[2] < 1)
        check(x, settings, gen, probs=True)


def test_extreme_settings_and_numbers():
    gen = torch.Generator().manual_seed(9)
    x = logits_of(gen, 12, 777, torch.float32)
    nan, inf = math.nan, math.inf
    best = x.argmax(1).tolist()

    def run(u, **kw):
        kw = {n: torch.tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32).cuda() for n, v in kw.items()}
        ids, probs = api.sample(x[:len(u)].cuda(), torch.tensor(u).cuda(), return_probs=True, **kw)
        return ids.cpu().tolist(), probs.cpu().double()

    ids, p = run([0.5] * 4, temperature=[0.0, -1.0, nan, 1e-30])  # greedy, and as good as
    assert ids == best[:4] and (p.amax(1) == 1).all()
    ids, p = run([0.123] * 2, temperature=[inf, 1e30])            # even
    assert ids == [int(0.123 * 777)] * 2 and ((p - 1 / 777).abs() < 1e-9).all()
    _, p = run([0.5] * 5, top_p=[nan, 2.0, 1.0, -3.0, 0.0])
    assert (p[:3] > 0).all() and ((p[3:] > 0).sum(1) == 1).all()
    _, p = run([0.5] * 4, min_p=[nan, -1.0, 0.0, 5.0])
    assert (p[:3] > 0).all() and (p[3] > 0).sum() == 1
    _, p = run([0.5] * 5, top_k=[-4, 0, 777, 2**31 - 1, 776])
    assert (p[:4] > 0).all() and (p[4] > 0).sum() == 776
    low, high = ([int(i) for i in (x[r] > -inf).nonzero()[[0, -1]]] for r in (0, 1))
    ids, _ = run([nan, -0.5, 0.0, 1.0, inf, 7.0, 1 - 2.0**-24])
    assert ids[:3] == [0, 0, 0] and ids[3:6] == [776] * 3
    assert low[0] == 0 and high[1] == 776


def test_outputs_streams_and_graphs():
    gen = torch.Generator().manual_seed(11)
    x, u = logits_of(gen, 5, 10007, torch.bfloat16).cuda(), torch.rand(5, generator=gen).cuda()
    want, p = api.sample(x, u, top_p=0.9, return_probs=True)
    out, room = torch.full((5,), -9, dtype=torch.int64, device="cuda"), torch.full((6, 10011), 7.0, device="cuda")
    assert api.sample(x, u, top_p=0.9, out=out, probs=room[:5, 2:10009]) is out
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(room[:5, 2:10009], p)
    assert (room[5] == 7.0).all() and (room[:, :2] == 7.0).all() and (room[:, 10009:] == 7.0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.sample(x, u, top_p=0.9, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # captured, and replayed on other numbers
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.sample(x, u, top_p=0.9, out=out)
    x2, u2 = logits_of(gen, 5, 10007, torch.bfloat16).cuda(), torch.rand(5, generator=gen).cuda()
    x.copy_(x2)
    u.copy_(u2)
    for _ in range(3):
        out.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, api.sample(x2, u2, top_p=0.9))
    # a row read by all (stride 0), and none at all
    same = api.sample(x[:1].expand(64, -1), torch.linspace(0, 0.99, 64).cuda(), temperature=1.2)
    assert same.unique().numel() > 1
    assert api.sample(x[:0], u[:0]).shape == (0,)


def test_many_calls_at_once():
    gen = torch.Generator().manual_seed(12)
    work = [(logits_of(gen, 7, 20000 + i, torch.float32).cuda(), torch.rand(7, generator=gen).cuda()) for i in range(6)]
    want = [api.sample(x, u, top_p=0.8, temperature=1.4) for x, u in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [api.sample(x, u, top_p=0.8, temperature=1.4, stream=s) for (x, u), s in zip(work, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_tensor_for_autograd_has_no_history():
    x = torch.randn(2, 50, device="cuda", requires_grad=True)
    ids, probs = api.sample(x, torch.rand(2, device="cuda"), return_probs=True)
    assert not probs.requires_grad and ids.shape == (2,)


# ---- judging ----

def judge(gen, counts, vocab, dtype, settings, *, drawn, scalar=False, strided=0, bad=(), mask=False):
    """Random drafts, against the reference; returns the accepted counts."""
    seqs, total = len(counts), sum(counts)
    rows = total + seqs
    target = logits_of(gen, rows, vocab, torch.float32)
    judged = [r for r in range(rows) if r not in {sum(counts[:i + 1]) + i for i in range(seqs)}]
    other = target[judged] * 0.95 + torch.randn((total, vocab), generator=gen) * 0.4
    q = torch.softmax(other, 1)
    drafts = (torch.multinomial(q, 1, generator=gen)[:, 0] if drawn else other.argmax(1)) if total else torch.zeros(0, dtype=torch.int64)
    for at, x in bad:
        drafts[at] = x
    if mask:
        target[:, ::4] = -math.inf
    logits = target.to(dtype)
    host = logits.double().numpy()
    of = [i for i, c in enumerate(counts) for _ in range(c + 1)]
    per = [settings] * seqs if scalar else settings
    p = [ref.distribution(host[r], f32(per[of[r]][0]), per[of[r]][1], f32(per[of[r]][2]), f32(per[of[r]][3])) for r in range(rows)]
    u = torch.rand((rows, 2), generator=gen).numpy()
    qn = q.numpy()
    for r in range(rows):  # numbers away from the borders
        u[r, 1] = away(p[r], u[r, 1])
        if r in judged:
            d = judged.index(r)
            x = int(drafts[d])
            if 0 <= x < vocab:
                rest = np.maximum(p[r] - qn[d], 0) if drawn else np.where(np.arange(vocab) == x, 0, p[r])
                if rest.sum() > 0:
                    u[r, 1] = away(rest, u[r, 1])
                edge = p[r][x] / (qn[d][x] if drawn else 1.0)
                if abs(u[r, 0] - edge) < CLOSE:
                    u[r, 0] *= np.float32(0.99)
    cu = [sum(counts[:i]) for i in range(seqs + 1)]
    if scalar:
        kw = dict(zip(("temperature", "top_k", "top_p", "min_p"), settings))
    else:
        t, k, tp, m = zip(*settings)
        kw = dict(temperature=torch.tensor(t, dtype=torch.float32).cuda(), top_k=torch.tensor(k, dtype=torch.int32).cuda(),
                  top_p=torch.tensor(tp, dtype=torch.float32).cuda(), min_p=torch.tensor(m, dtype=torch.float32).cuda())
    x, probs = logits.cuda(), q.cuda()
    if strided:
        wide = torch.full((rows, vocab + strided), math.nan, dtype=dtype, device="cuda")
        wide[:, 1:1 + vocab] = x
        x = wide[:, 1:1 + vocab]
        wide = torch.full((total, vocab + strided), math.nan, device="cuda")
        wide[:, 2:2 + vocab] = probs
        probs = wide[:, 2:2 + vocab]
    ids, accepted = api.verify_drafts(x, drafts.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), torch.from_numpy(u).cuda(),
                                      draft_probs=probs if drawn else None, **kw)
    ids, accepted = ids.cpu().tolist(), accepted.cpu().tolist()
    for s, n in enumerate(counts):
        a = cu[s] + s
        want, taken = ref.verify(p[a:a + n + 1], drafts[cu[s]:cu[s + 1]].tolist(), u[a:a + n + 1], qn[cu[s]:cu[s + 1]] if drawn else None)
        assert ids[a:a + n + 1] == want and accepted[s] == taken, (s, ids[a:a + n + 1], want)
    return accepted


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("setting", [(1.0, 0, 1.0, 0.0), (0.8, 20, 0.95, 0.02), (1.2, 0, 0.9, 0.0), (0.0, 0, 1.0, 0.0)])
def test_judging(setting, dtype, drawn):
    gen = torch.Generator().manual_seed(21)
    taken = judge(gen, [7, 0, 3, 15, 1, 40, 2], 1500, TYPES[dtype], setting, drawn=drawn, scalar=True, strided=5)
    if setting[0] > 0 and drawn:
        assert 0 < sum(taken) < 68


@pytest.mark.parametrize("drawn", [True, False])
def test_judging_with_settings_of_their_own(drawn):
    gen = torch.Generator().manual_seed(22)
    counts = [3] * len(SETTINGS)
    judge(gen, counts, 4099, torch.float32, SETTINGS, drawn=drawn, mask=True)


@pytest.mark.parametrize("drawn", [True, False])
def test_judging_large_vocabularies(drawn):
    gen = torch.Generator().manual_seed(23)
    for dtype, setting in ((torch.float32, (1.0, 0, 1.0, 0.0)), (torch.bfloat16, (0.7, 0, 0.9, 0.0)), (torch.float16, (1.0, 50, 1.0, 0.0))):
        judge(gen, [5, 2], 151936, dtype, setting, drawn=drawn, scalar=True)


def test_drafts_that_are_none_and_sequences_without_any():
    gen = torch.Generator().manual_seed(24)
    taken = judge(gen, [4, 4, 0, 0, 2], 900, torch.float32, (1.0, 0, 1.0, 0.0), drawn=True, scalar=True, bad=[(0, -1), (5, 900), (8, 2**40)])
    assert taken[0] == 0 and taken[1] <= 1 and taken[4] == 0
    judge(gen, [0, 0, 0], 900, torch.float32, (1.0, 0, 1.0, 0.0), drawn=False, scalar=True)
    judge(gen, [0] * 1300, 40, torch.float32, (1.0, 0, 1.0, 0.0), drawn=False, scalar=True)


def test_judging_many_sequences():
    """More sequences than a row's own is looked for among at a time, of none to three drafts, each with its settings; then rows behind them
    and a last sequence whose end is out of range."""
    gen = torch.Generator().manual_seed(29)
    for seqs in (33, 64, 1025):
        settings = [SETTINGS[i % len(SETTINGS)] for i in range(seqs)]
        judge(gen, [(i * 7 + i // 5) % 4 for i in range(seqs)], 40, torch.float32, settings, drawn=seqs % 2 == 0)
    seqs = 1100
    cu = torch.arange(0, 2 * seqs + 1, 2, dtype=torch.int32)
    cu[-1] = 4 * seqs
    x = torch.randn((4 * seqs, 50), generator=gen).cuda()
    drafts = torch.zeros(3 * seqs, dtype=torch.int64)
    drafts[:2 * seqs] = x.cpu().view(-1, 50)[torch.arange(3 * seqs).view(seqs, 3)[:, :2].reshape(-1)].argmax(1)
    ids, taken = torch.full((4 * seqs,), -77).cuda(), torch.full((seqs,), -77, dtype=torch.int32).cuda()
    api.verify_drafts(x, drafts.cuda(), cu.cuda(), torch.zeros((4 * seqs, 2)).cuda(), temperature=0.0, out=ids, accepted=taken)
    assert taken.tolist() == [2] * (seqs - 1) + [-77]
    assert (ids[3 * (seqs - 1):] == -77).all() and torch.equal(ids[:3 * (seqs - 1)], x[:3 * (seqs - 1)].argmax(1))


def test_special_distributions():
    """The draft's distribution is the target's (all accepted), misses it altogether (none), and rows without tokens."""
    vocab, k = 333, 6
    x = torch.randn((k + 1, vocab), generator=torch.Generator().manual_seed(25)).cuda()
    u = torch.full((k + 1, 2), 0.999, device="cuda")
    cu = torch.tensor([0, k], dtype=torch.int32).cuda()
    drafts, p = api.sample(x[:k], torch.linspace(0, 0.9, k).cuda(), return_probs=True)
    ids, n = api.verify_drafts(x, drafts, cu, u, draft_probs=p)
    assert n.tolist() == [k] and torch.equal(ids[:k], drafts) and ids[k] >= 0
    # q of one token that the target never takes
    masked = x.clone()
    masked[:, 17] = -math.inf
    q = torch.zeros((k, vocab), device="cuda")
    q[:, 17] = 1.0
    ids, n = api.verify_drafts(masked, torch.full((k,), 17, device="cuda"), cu, u, draft_probs=q)
    assert n.tolist() == [0] and ids[0] == api.sample(masked[:1], u[:1, 1].contiguous())[0] and (ids[1:] == -1).all()
    # the target's only token is the draft: accepted whatever the number
    one = torch.full_like(x, -math.inf)
    one[:, 5] = 0.0
    ids, n = api.verify_drafts(one, torch.full((k,), 5, device="cuda"), cu, u)
    assert n.tolist() == [k] and (ids == 5).all()
    # nothing left of the first row: no draft is accepted and none drawn
    none = x.clone()
    none[0] = -math.inf
    ids, n = api.verify_drafts(none, drafts, cu, u, draft_probs=p)
    assert n.tolist() == [0] and (ids == -1).all()
    # what remains is nothing though the draft is refused: drawn from the target itself
    over = p.clone().mul_(2.0)
    ids, n = api.verify_drafts(x, drafts, cu, u, draft_probs=over)
    assert n.tolist() == [0] and ids[0] == api.sample(x[:1], u[:1, 1].contiguous())[0]


def test_rows_of_no_sequence_are_left_as_they_are():
    gen = torch.Generator().manual_seed(26)
    x, u = torch.randn((20, 100), generator=gen).cuda(), torch.rand((20, 2), generator=gen).cuda()
    drafts = torch.randint(0, 100, (17,), generator=gen).cuda()
    for bounds, covered in (([0, 4, 6, 9], 12), ([0, 4, 2, 6], None), ([0, 5, 40, 17], None), ([-3, 2, 4, 5], None), ([9, 1, 0, 17], None)):
        out = torch.full((20,), -77, dtype=torch.int64, device="cuda")
        taken = torch.full((3,), -77, dtype=torch.int32, device="cuda")
        api.verify_drafts(x, drafts, torch.tensor(bounds, dtype=torch.int32).cuda(), u, out=out, accepted=taken)
        torch.cuda.synchronize()
        if covered:
            assert (out[covered:] == -77).all() and (out[:covered] != -77).all() and (taken >= 0).all()
        else:  # a sequence out of range is passed over
            good = [0 <= a <= b <= 17 for a, b in zip(bounds, bounds[1:])]
            assert [t != -77 for t in taken.tolist()] == good


def test_judging_in_a_graph_and_on_a_stream():
    gen = torch.Generator().manual_seed(27)
    x, u = torch.randn((24, 5000), generator=gen).cuda(), torch.rand((24, 2), generator=gen).cuda()
    drafts = x.argmax(1)[:21].contiguous()
    cu = torch.tensor([0, 7, 14, 21], dtype=torch.int32).cuda()
    want = api.verify_drafts(x, drafts, cu, u, temperature=0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.verify_drafts(x, drafts, cu, u, temperature=0.9, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, taken = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.verify_drafts(x, drafts, cu, u, temperature=0.9, out=out, accepted=taken)
    u.copy_(torch.rand((24, 2), generator=gen))
    for _ in range(2):
        out.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        again = api.verify_drafts(x, drafts, cu, u, temperature=0.9)
        assert torch.equal(out, again[0]) and torch.equal(taken, again[1])


def test_drawn_and_judged_together():
    """A cycle: drafts drawn one position after another with their distributions, then judged; every token comes from the target's set."""
    gen = torch.Generator().manual_seed(28)
    seqs, k, vocab = 5, 4, 2000
    target = logits_of(gen, seqs * (k + 1), vocab, torch.float16).cuda()
    settings = dict(temperature=0.8, top_k=20, top_p=0.9)
    rows = torch.arange(seqs * (k + 1)).view(seqs, k + 1)[:, :k].reshape(-1).cuda()
    drafter = (target.float()[rows] + torch.randn((seqs * k, vocab), generator=gen).cuda() * 0.3).contiguous()
    drafts, q = api.sample(drafter, torch.rand(seqs * k, generator=gen).cuda(), return_probs=True, **settings)
    u = torch.rand((seqs * (k + 1), 2), generator=gen).cuda()
    ids, n = api.verify_drafts(target, drafts, torch.arange(0, seqs * k + 1, k, dtype=torch.int32).cuda(), u, draft_probs=q, **settings)
    _, p = api.sample(target, u[:, 0].contiguous(), return_probs=True, **settings)
    for s in range(seqs):
        a = int(n[s])
        for i in range(k + 1):
            token = int(ids[s * (k + 1) + i])
            assert (token == -1) == (i > a)
            if token >= 0:
                assert p[s * (k + 1) + i, token] > 0
                assert i == a or token == int(drafts[s * k + i])
