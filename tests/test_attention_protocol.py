"""Host model check of the paged-attention kernel's pipeline (csrc/paged_attention.cu): the copying warp, the MMA
warp, the two softmax groups and what they start asynchronously (copies that land in any order, tensor-core batches in
order, with their commits) run over random interleavings.  Barriers are modelled with their
phases: a wait tests a parity, as the hardware does, and the model checks that the phase it meant has really completed --
a parity passes too early when a barrier is two phases behind.  Buffers are checked for every read and write."""
import random

import pytest

MODES = {  # name: (query tiles share keys, ring entries)
    "pair_128": (True, 5), "single_128": (False, 6), "pair_64": (True, 12), "single_64": (False, 13)}


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase, self.tx = count, count, 0, 0

    def _turn(self):
        if self.left == 0 and self.tx == 0:
            self.phase += 1
            self.left = self.count

    def arrive(self, tx=0):
        assert self.left > 0, "arrival beyond the count"
        self.tx += tx
        self.left -= 1
        self._turn()

    def land(self, tx):
        self.tx -= tx
        assert self.tx >= 0
        self._turn()

    def test(self, n):
        """Whether the parity test for phase n passes; it must not pass before the phase is complete."""
        passes = self.phase & 1 != n & 1
        assert not passes or self.phase > n, "a parity test passed for a phase that is not complete"
        assert self.phase <= n + 1, "a phase was left behind"
        return passes


class Model:
    def __init__(self, mode, segments, rng):
        self.pair, self.stages = MODES[mode]
        self.segments, self.rng = segments, rng
        self.edges = [{t for t in range(nt) if t in (0, nt - 1) or rng.random() < 0.3} for nt in segments]
        b = self.b = {}
        for i in range(self.stages):
            b["full", i], b["empty", i] = Bar(1), Bar(1)
        b["q_full"], b["q_empty"] = Bar(1), Bar(1)
        for s in range(2):
            for name in ("s_full", "p_half", "p_ready", "o_full"):
                b[name, s] = Bar(1)
        b["sync"] = Bar(2)
        self.ring = [None] * self.stages
        self.q = None
        self.S = [None] * 2        # of each stream: its scores, then its weights in the same place
        self.O = [None] * 2        # list of tiles added, or "read"
        self.copies = []           # landing in any order
        self.queue = []
        self.results = []

    # ---- roles: generators that yield a barrier and phase to wait for, or None ----
    def loader(self):
        put = 0
        for g, nt in enumerate(self.segments):
            if g:
                yield "q_empty", g - 1
            assert self.q is None or self.q[1] == 0
            self.b["q_full"].arrive(tx=1)
            self.copies.append(("q_full", 1, lambda g=g, nt=nt: setattr(self, "q", [g, nt if not self.pair else 2 * nt])))
            for t in range(nt):
                for kind in "kv":
                    st = put % self.stages
                    if put >= self.stages:
                        yield ("empty", st), put // self.stages - 1
                    self.b["full", st].arrive(tx=1)
                    assert self.ring[st] is None, "a slot is filled before it is free"
                    self.copies.append((("full", st), 1, lambda st=st, v=[kind, g, t]: self.ring.__setitem__(st, v)))
                    put += 1
                    yield None
        for p in range(max(0, put - self.stages), put):
            yield ("full", p % self.stages), p // self.stages

    def order(self, nt):
        for t in range(nt):
            for s in (range(2) if self.pair else (t & 1,)):
                yield t, s

    def mma(self):
        base, n = 0, [0, 0]

        def full(p):
            return ("full", p % self.stages), p // self.stages

        for g, nt in enumerate(self.segments):
            count = [nt, nt] if self.pair else [(nt + 1) // 2, nt // 2]
            p0, base = 2 * base, base + nt
            left = [nt * (2 if self.pair else 1)]

            def entry(s, i):
                return p0 + (2 * i if self.pair else 2 * (2 * i + s))

            def scores(s, i):
                p, t = entry(s, i), i if self.pair else 2 * i + s
                shared = self.pair and s == 0
                left[0] -= 1

                def work(g=g):
                    assert self.q[0] == g and self.ring[p % self.stages] == ["k", g, t], "the wrong keys"
                    assert self.S[s] is None, "weights that were not used are overwritten"
                    self.S[s] = ("scores", g, t)
                    self.q[1] -= 1
                    if not shared:
                        self.ring[p % self.stages] = None
                self.queue.append((work, [("s_full", s)] + ([] if shared else [("empty", p % self.stages)]) +
                                   (["q_empty"] if left[0] == 0 else [])))

            def values(s, i, half):
                p, t = entry(s, i) + 1, i if self.pair else 2 * i + s
                shared = self.pair and s == 0

                def work(g=g):
                    assert self.ring[p % self.stages] == ["v", g, t], "the wrong values"
                    assert self.S[s] in (("half", g, t), ("weights", g, t)) and (half == 0 or self.S[s][0] == "weights")
                    if half == 0:
                        if i == 0:
                            assert self.O[s] in (None, "read"), "an output that was not read is overwritten"
                            self.O[s] = []
                        return
                    self.O[s].append((g, t))
                    self.S[s] = None
                    if not shared:
                        self.ring[p % self.stages] = None
                self.queue.append((work, [] if half == 0 else ([] if shared else [("empty", p % self.stages)]) +
                                   ([("o_full", s)] if i + 1 == count[s] else [])))

            yield "q_full", g
            for s in range(2):
                if count[s]:
                    if s == 0 or not self.pair:
                        yield full(entry(s, 0))
                    scores(s, 0)
                    yield None
            for i in range(count[0]):
                for s in range(2):
                    if i >= count[s]:
                        continue
                    more = i + 1 < count[s]
                    if s == 0 or not self.pair:
                        yield full(entry(s, i) + 1)
                        if self.pair and more:
                            yield full(entry(s, i + 1))
                    yield ("p_half", s), n[s]
                    values(s, i, 0)
                    yield None
                    yield ("p_ready", s), n[s]
                    n[s] += 1
                    values(s, i, 1)
                    if more:
                        if not self.pair:
                            yield None
                            yield full(entry(s, i + 1))
                        scores(s, i + 1)
                    yield None

    def softmax(self, s):
        tile, segs, sync, base = 0, [0, 0], 0, 0
        for g, nt in enumerate(self.segments):
            mine = [t for t, u in self.order(nt) if u == s]
            for i, t in enumerate(mine):
                yield ("s_full", s), tile
                tile += 1
                if t in self.edges[g]:  # values that no row sees are cleared
                    p = 2 * (base + t) + 1
                    yield ("full", p % self.stages), p // self.stages
                    assert self.ring[p % self.stages] == ["v", g, t]
                assert self.S[s] == ("scores", g, t)
                # O may be rescaled here: the second products before these scores are done
                assert i == 0 or self.O[s][-1] == (g, mine[i - 1])
                self.S[s] = ("half", g, t)
                self.b["p_half", s].arrive()
                yield None
                self.S[s] = ("weights", g, t)
                self.b["p_ready", s].arrive()
                yield None
            base += nt
            for u in ((s,) if self.pair else (0, 1)):
                if self.pair or nt > u:
                    yield ("o_full", u), segs[u]
                    segs[u] += 1
                    assert self.O[u] == [(g, t) for t, v in self.order(nt) if v == u]
            if self.pair:
                self.O[s] = "read"
            else:  # both groups meet to exchange their sums, read both outputs, and meet again
                self.b["sync"].arrive()
                yield "sync", sync
                sync += 1
                reading = [nt > 0, nt > 1]
                assert all(not r or isinstance(o, list) for r, o in zip(reading, self.O))
                self.b["sync"].arrive()
                yield "sync", sync
                sync += 1
                self.O[s] = "read" if reading[s] else self.O[s]
            self.results.append((g, s))

    def run(self):
        roles = {"loader": self.loader(), "mma": self.mma(), "s0": self.softmax(0), "s1": self.softmax(1)}
        waits = dict.fromkeys(roles)
        slow = self.rng.choice(list(roles) + ["copies", "tensor", None])  # one party that is rarely served
        idle = 0
        while roles:
            choices = list(roles) + (["copies"] if self.copies else []) + (["tensor"] if self.queue else [])
            who = self.rng.choice(choices)
            if idle < 2000 and self.rng.random() < 0.95 and who == slow:
                idle += 1
                continue
            moved = True
            if who == "copies":
                bar, tx, put = self.copies.pop(self.rng.randrange(len(self.copies)))
                put()
                self.b[bar].land(tx)
            elif who == "tensor":
                work, commits = self.queue.pop(0)
                work()
                for c in commits:
                    self.b[c].arrive()
            else:
                w = waits[who]
                if w is not None and not self.b[w[0]].test(w[1]):
                    moved = False
                else:
                    try:
                        waits[who] = next(roles[who])
                    except StopIteration:
                        del roles[who], waits[who]
            idle = 0 if moved else idle + 1
            assert idle < 20000, f"no progress: {waits}"
        assert not self.copies and len(self.results) == 2 * len(self.segments)


@pytest.mark.parametrize("mode", list(MODES))
def test_every_interleaving_tried_is_sound(mode):
    for seed in range(150):
        rng = random.Random(seed)
        segments = [rng.choice([1, 1, 2, 3, 4, 5, 7, 12, 19]) for _ in range(rng.randint(1, 5))]
        Model(mode, segments, rng).run()


def test_the_model_catches_a_waiter_that_skips_phases():
    # One MMA role a stream, each waiting only for its own tiles: a slot's next phase is tested while the last one's copy
    # may still be under way.
    class PerStream(Model):
        def one(self, s):
            n = 0
            for g, nt in enumerate(self.segments):
                base = sum(self.segments[:g])
                for t in range(s, nt, 2):
                    p = 2 * (base + t)
                    yield ("full", p % self.stages), p // self.stages
                    yield ("full", (p + 1) % self.stages), (p + 1) // self.stages
                    for e in (p, p + 1):
                        self.b["empty", e % self.stages].arrive()
                        self.ring[e % self.stages] = None
                    n += 1
                    yield None

    def simulate(seed):
        rng = random.Random(seed)
        m = PerStream("single_128", [40], rng)
        roles = [m.one(0), m.one(1), m.loader()]
        waits = [None] * 3
        m.b["q_empty"].arrive()
        for _ in range(40000):
            if m.copies and rng.random() < 0.2:
                bar, tx, put = m.copies.pop(rng.randrange(len(m.copies)))
                put()
                m.b[bar].land(tx)
            i = rng.randrange(3)
            if roles[i] is None or (waits[i] is not None and not m.b[waits[i][0]].test(waits[i][1])):
                continue
            try:
                waits[i] = next(roles[i])
            except StopIteration:
                roles[i] = None

    with pytest.raises(AssertionError):
        for seed in range(50):
            simulate(seed)
