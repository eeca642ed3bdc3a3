"""From logits to kept tokens, measured: drawing tokens with temperature, top-k, top-p and min-p, judging
drafted tokens against the target's logits, and the attention of new tokens over a paged cache of which they
see a window and the row's first tokens.

Each case is one call as a serving loop makes it.  ``own`` selects the library's kernels; otherwise ``run``
computes the same thing from elementary torch operations: in 32 bits for the attention, in 64 where a draw or
a nucleus has to fall on the right side of a border.

Random numbers are inputs.  A row's order of tokens is logit descending, index ascending.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- the cases ---------------------------------------------------------------------------
def listed():
    heads = dict(q_heads=32, kv_heads=8, head_dim=128)
    return [
        # one user's next token with a chat's usual settings: latency is all of it
        dict(name="sample_one_row", op="sample", rows=1, vocab=151936, dtype="fp32", temperature=0.8, top_k=50, top_p=0.95,
             min_p=0.0, mixed=False, probs=False, mask="none", spread=2.0, salt=1),
        # the requests of a small model's batch, each with settings of its own, padded vocabulary entries masked
        dict(name="sample_batch_mixed", op="sample", rows=24, vocab=32000, dtype="fp16", temperature=0.9, top_k=40, top_p=0.9,
             min_p=0.05, mixed=True, probs=False, mask="tail", spread=2.0, salt=2),
        # four requests' drafts of seven positions: the distribution is wanted too, for the verification
        dict(name="sample_drafts_probs", op="sample", rows=28, vocab=151936, dtype="fp32", temperature=1.0, top_k=0, top_p=0.9,
             min_p=0.0, mixed=False, probs=True, mask="none", spread=2.0, salt=3),
        # many samples at a high temperature: wide nuclei, tens of thousands of tokens
        dict(name="sample_wide_nucleus", op="sample", rows=96, vocab=151936, dtype="bf16", temperature=1.6, top_k=0, top_p=0.97,
             min_p=0.0, mixed=False, probs=False, mask="none", spread=3.0, salt=4),
        # a rollout of many sequences from the whole distribution: the logits' bytes bound it
        dict(name="sample_whole_large", op="sample", rows=256, vocab=248320, dtype="bf16", temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, mixed=False, probs=False, mask="tail", spread=2.0, salt=5),
        # one request's seven greedily drafted tokens
        dict(name="verify_one", op="verify", seqs=1, lo=7, hi=7, vocab=151936, dtype="fp32", temperature=0.7, top_k=0, top_p=0.9,
             min_p=0.0, mixed=False, drawn=False, mask="none", spread=2.0, salt=6),
        # a ragged batch whose drafts were drawn, some requests without any, settings of their own
        dict(name="verify_batch_mixed", op="verify", seqs=16, lo=0, hi=7, vocab=32000, dtype="fp16", temperature=0.9, top_k=30,
             top_p=0.95, min_p=0.02, mixed=True, drawn=True, mask="tail", spread=2.0, salt=7),
        # eight requests, fifteen drawn drafts each over the full vocabulary, from the whole distribution
        dict(name="verify_full_vocab", op="verify", seqs=8, lo=15, hi=15, vocab=248320, dtype="fp32", temperature=1.0, top_k=0,
             top_p=1.0, min_p=0.0, mixed=False, drawn=True, mask="none", spread=2.0, salt=8),
        # one user's next token far into a long document, the drafter's view of it
        dict(name="sinks_one_token", op="attention", **heads, dtype="bf16", page=16, seqs=1, new_lo=1, new_hi=1, ctx_lo=50000,
             ctx_hi=50000, causal=True, window=1024, sinks=4, salt=9),
        # draft blocks of seven positions for 16 ragged requests that see each other, sinks that end inside a page
        dict(name="sinks_draft_block", op="attention", **heads, dtype="bf16", page=16, seqs=16, new_lo=7, new_hi=7, ctx_lo=300,
             ctx_hi=30000, causal=False, window=2048, sinks=20, salt=10),
        # a decode batch of a small model, 7 query heads to a kv head
        dict(name="sinks_decode_batch", op="attention", q_heads=28, kv_heads=4, head_dim=64, dtype="fp16", page=64, seqs=64,
             new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=20000, causal=True, window=4000, sinks=64, salt=11),
        # a long prompt's last quarter
        dict(name="sinks_prompt_chunk", op="attention", **heads, dtype="bf16", page=64, seqs=1, new_lo=4096, new_hi=4096,
             ctx_lo=12288, ctx_hi=12288, causal=True, window=4096, sinks=128, salt=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "verify", "attention"])
    salt = rng.randrange(1, 1 << 30)
    if op == "attention":
        dim, kv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 7, 8])
        seqs, ctx = _log(rng, 1, 48), _log(rng, 1, 60000)
        new = rng.choice([1, _log(rng, 1, 16), _log(rng, 16, 4000)])
        while seqs > 1 and (seqs * new * (new + ctx) * kv * group > 2e9 or seqs * (ctx + new) * kv * dim > 2e8):
            seqs, ctx = max(1, seqs // 2), max(1, ctx // 2)
        while new * (new + ctx) * kv * group > 2e9:
            new = max(1, new // 2)
        return dict(op=op, q_heads=kv * group, kv_heads=kv, head_dim=dim, dtype=rng.choice(["bf16", "fp16"]),
                    page=rng.choice([16, 32, 64, 128]), seqs=seqs, new_lo=max(1, new // rng.choice([1, 1, 3])), new_hi=new,
                    ctx_lo=rng.choice([0, ctx // 3, ctx]), ctx_hi=ctx, causal=rng.random() < 0.75, window=_log(rng, 5, 6000),
                    sinks=rng.choice([1, 4, _log(rng, 1, 700)]), salt=salt)
    vocab = rng.choice([4096, 32000, 151936, 248320, _log(rng, 500, 248320), _log(rng, 500, 248320)])
    rows = min(_log(rng, 1, 300), max(1, 40_000_000 // vocab))
    some = dict(vocab=vocab, dtype=rng.choice(["bf16", "fp16", "fp32"]), temperature=round(rng.uniform(0.3, 1.7), 3),
                top_k=rng.choice([0, 0, _log(rng, 1, 100), _log(rng, 1, 3000)]), top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)]), mixed=rng.random() < 0.4,
                mask=rng.choice(["none", "tail", "grammar"]), spread=round(rng.uniform(1.0, 3.0), 2), salt=salt)
    if op == "sample":
        return dict(op=op, rows=rows, probs=rng.random() < 0.4, **some)
    hi = rng.choice([1, 3, 7, 15])
    return dict(op=op, seqs=max(1, rows // (hi + 1)), lo=rng.choice([0, hi]), hi=hi, drawn=rng.random() < 0.6, **some)


# ---- what a case's sizes are --------------------------------------------------------------
def _spread(case, lo, hi, n, tag):
    """n whole numbers from lo to hi; lo and hi are among them where n allows."""
    r = random.Random("%d %s" % (case["salt"], tag))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[0] = hi
    if n > 1:
        v[-1] = lo
    return v


def _lengths(case):
    """(new tokens, tokens before them) of each sequence."""
    n = case["seqs"]
    return _spread(case, case["new_lo"], case["new_hi"], n, "new"), _spread(case, case["ctx_lo"], case["ctx_hi"], n, "ctx")


def _drafts(case):
    return _spread(case, case["lo"], case["hi"], case["seqs"], "drafts")


def _settings(case):
    """Temperature, top-k, top-p and min-p of each row (sample) or sequence (verify)."""
    n = case["rows"] if case["op"] == "sample" else case["seqs"]
    base = (case["temperature"], case["top_k"], case["top_p"], case["min_p"])
    if not case["mixed"]:
        return [list(v) for v in zip(*[base] * n)]
    r = random.Random("%d settings" % case["salt"])
    rows = []
    for _ in range(n):  # greedy ones, ones with the case's settings and ones that leave some of them off among them
        t, k, p, m = base
        t = r.choice([t, t, 0.0, round(t * r.uniform(0.5, 1.5), 3)])
        rows.append((t, r.choice([k, 0, r.randint(1, 200)]), r.choice([p, 1.0, round(r.uniform(0.2, 0.99), 3)]), r.choice([m, 0.0])))
    return [list(v) for v in zip(*rows)]


def work(case):
    if case["op"] == "attention":
        new, ctx = _lengths(case)
        pairs = keys = 0
        for n, c in zip(new, ctx):
            length, first = n + c, max(0, c - case["window"] + 1)
            for i in range(n):
                hi, lo = (c + i + 1 if case["causal"] else length), max(0, c + i - case["window"] + 1)
                pairs += hi - lo + min(lo, case["sinks"])
            keys += length - first + min(first, case["sinks"])
        row = case["head_dim"] * 2
        rows = sum(new) * case["q_heads"]
        return {"bytes": 2 * rows * row + rows * 4 + 2 * keys * case["kv_heads"] * row,
                "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}
    size = SIZES[case["dtype"]]
    if case["op"] == "sample":
        entries = case["rows"] * case["vocab"]
        return {"bytes": entries * (size + (4 if case["probs"] else 0)) + 12 * case["rows"], "flops": 3 * entries}
    drafts = _drafts(case)
    rows, some = sum(drafts) + case["seqs"], sum(1 for d in drafts if d)
    # of the drafts' distributions a draw needs the rejected one's
    return {"bytes": rows * (case["vocab"] * size + 16) + (4 * some * case["vocab"] if case["drawn"] else 0),
            "flops": 3 * rows * case["vocab"]}


# ---- inputs -------------------------------------------------------------------------------
def _logits(case, rows, gen):
    """Logits as a model gives them: most tokens in a broad bell, a few hundred that fit well above it."""
    x = torch.randn((rows, case["vocab"]), generator=gen, device="cuda") * case["spread"]
    n = min(300, case["vocab"] // 3)
    at = torch.randint(0, case["vocab"], (rows, n), generator=gen, device="cuda")
    return x.scatter_add_(1, at, torch.randn((rows, n), generator=gen, device="cuda").abs_().mul_(3.0).add_(2.0))


def _masked(case, x, gen):
    rows, vocab = x.shape
    if case["mask"] == "tail":  # entries that pad the vocabulary
        x[:, vocab - max(1, vocab // 300):] = float("-inf")
    elif case["mask"] == "grammar":  # a row's next token is one of a few
        allowed = torch.randint(0, vocab, (rows, 40), generator=gen, device="cuda")
        y = torch.full_like(x, float("-inf"))
        x = y.scatter_(1, allowed, x.gather(1, allowed))
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + case["salt"])
    s = {"case": case}
    dtype = TYPES[case["dtype"]]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if case["op"] == "attention":
        new, ctx = _lengths(case)
        page, tokens = case["page"], [n + c for n, c in zip(new, ctx)]
        wide, used, table = max(-(-t // page) for t in tokens), 0, []
        for t in tokens:
            n = -(-t // page)
            table.append(list(range(used, used + n)) + [-1] * (wide - n))
            used += n
        pages = used + 3
        # pages scattered over the pool as in a server that has run for a while
        order = torch.cat((torch.randperm(pages, generator=gen, device="cuda"), torch.full((1,), -1, device="cuda")))
        s["pool"] = torch.randn((pages, 1, 2, case["kv_heads"], page, case["head_dim"]), generator=gen, device="cuda", dtype=dtype)
        s["table"] = order[torch.tensor(table, device="cuda")].to(torch.int32)
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        s["length"] = ints(tokens)
        s["max_new"] = max(new)
        s["cu_new"] = ints([sum(new[:i]) for i in range(len(new) + 1)])
        s["q"] = torch.randn((sum(new), case["q_heads"], case["head_dim"]), generator=gen, device="cuda", dtype=dtype)
        if own:  # the cache as a program keeps it
            from dspark_draft_sampling_gb300 import api

            s["cache"] = api.PagedCache(s["pool"], s["table"], s["length"], s["refs"])
        return s
    t, k, p, m = _settings(case)
    s["settings"] = {"temperature": torch.tensor(t, dtype=torch.float32, device="cuda"), "top_k": ints(k),
                     "top_p": torch.tensor(p, dtype=torch.float32, device="cuda"),
                     "min_p": torch.tensor(m, dtype=torch.float32, device="cuda")}
    if case["op"] == "sample":
        s["logits"] = _masked(case, _logits(case, case["rows"], gen), gen).to(dtype)
        s["uniforms"] = torch.rand(case["rows"], generator=gen, device="cuda")
        return s
    drafts = _drafts(case)
    rows, total = sum(drafts) + case["seqs"], sum(drafts)
    target = _logits(case, rows, gen)
    judged = torch.ones(rows, dtype=torch.bool, device="cuda")  # all rows but each sequence's last
    judged[torch.cumsum(torch.tensor(drafts, device="cuda") + 1, 0) - 1] = False
    # the drafter's view of the same positions: alike, not equal
    other = target[judged] * 0.95
    other += torch.randn(other.shape, generator=gen, device="cuda") * 0.5
    if case["drawn"]:
        q = torch.softmax(other, 1)
        s["draft_probs"] = q
        s["drafts"] = torch.multinomial(q, 1, generator=gen)[:, 0] if total else torch.zeros(0, dtype=torch.int64, device="cuda")
    else:
        s["draft_probs"] = None
        s["drafts"] = other.argmax(1) if total else torch.zeros(0, dtype=torch.int64, device="cuda")
    s["logits"] = _masked(case, target, gen).to(dtype)
    s["cu_drafts"] = ints([sum(drafts[:i]) for i in range(len(drafts) + 1)])
    s["uniforms"] = torch.rand((rows, 2), generator=gen, device="cuda")
    return s


# ---- one pass -----------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _given(s):
    """The settings as a call takes them: one number for all where the case says so."""
    c = s["case"]
    return s["settings"] if c["mixed"] else {n: c[n] for n in ("temperature", "top_k", "top_p", "min_p")}


def _own_sample(s):
    from dspark_draft_sampling_gb300 import api

    if s["case"]["probs"]:
        ids, probs = api.sample(s["logits"], s["uniforms"], return_probs=True, **_given(s))
        return {"ids": ids, "probs": probs}
    return {"ids": api.sample(s["logits"], s["uniforms"], **_given(s))}


def _own_verify(s):
    from dspark_draft_sampling_gb300 import api

    ids, accepted = api.verify_drafts(s["logits"], s["drafts"], s["cu_drafts"], s["uniforms"], draft_probs=s["draft_probs"], **_given(s))
    return {"ids": ids, "accepted": accepted}


def _own_attention(s):
    from dspark_draft_sampling_gb300 import api

    c = s["case"]
    out, lse = api.paged_attention(s["q"], s["cache"], 0, s["cu_new"], max_new=s["max_new"], causal=c["causal"], window=c["window"],
                                   sinks=c["sinks"], return_lse=True)
    return {"out": out, "lse": lse}


# ---- the plain forms ----------------------------------------------------------------------
def _weights(logits, settings, plain):
    """What each token of each row weighs in a draw, in index order and 64 bits; 0 for what the settings drop.
    plain: no row has a setting that drops tokens."""
    t, k, p, m = (settings[n][:, None] for n in ("temperature", "top_k", "top_p", "min_p"))
    t = t.double()
    if plain:
        x = logits.double()
        top = x.amax(1, keepdim=True)
        return x.sub_(torch.where(top == float("-inf"), 0.0, top)).div_(t).exp_()
    x, order = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    x = x.double()
    rank = torch.arange(x.shape[1], device=x.device)[None]
    some = x > float("-inf")
    top = torch.where(some[:, :1], x[:, :1], 0.0)
    w = ((x - top) / torch.where(t > 0, t, 1.0)).exp_()
    w = torch.where(some & ((k <= 0) | (rank < k)), w, 0.0)
    upto = torch.cumsum(w, 1)
    keep = (p >= 1) | (upto - w < p.double() * upto[:, -1:]) | (rank == 0)
    keep &= (w >= m.double()) & some
    keep &= (t > 0) | (rank == 0)
    w = torch.where(keep, w, 0.0)
    return torch.zeros_like(w).scatter_(1, order, w)


def _pick(w, u):
    """The lowest token whose weights up to it exceed u of the row's sum; -1 where nothing weighs anything."""
    upto = torch.cumsum(w, 1)
    total = upto[:, -1:]
    return torch.where(total[:, 0] > 0, (upto <= u[:, None].double() * total).sum(1), -1)


def _is_plain(case):
    return not case["mixed"] and case["top_k"] == 0 and case["top_p"] >= 1 and case["min_p"] == 0


def _plain_sample(s):
    w = _weights(s["logits"], s["settings"], _is_plain(s["case"]))
    ids = _pick(w, s["uniforms"])
    if not s["case"]["probs"]:
        return {"ids": ids}
    total = w.sum(1, keepdim=True)
    return {"ids": ids, "probs": (w / torch.where(total > 0, total, 1.0)).float()}


def _plain_verify(s):
    cu, drafts, logits, u = s["cu_drafts"].long(), s["drafts"], s["logits"], s["uniforms"]
    rows, seqs = logits.shape[0], cu.numel() - 1
    r = torch.arange(rows, device="cuda")
    ends = cu[1:] + torch.arange(1, seqs + 1, device="cuda")  # of each sequence's rows
    of = torch.searchsorted(ends, r, right=True)
    d = r - of  # the draft that the row judges
    judges = r != ends[of] - 1
    w = _weights(logits, {n: v[of] for n, v in s["settings"].items()}, _is_plain(s["case"]))
    total = w.sum(1)
    p = w / torch.where(total > 0, total, 1.0)[:, None]
    take = torch.zeros(rows, dtype=torch.bool, device="cuda")
    if drafts.numel():
        jr, x = r[judges], drafts[d[judges]]
        px = p[jr, x]
        rest = p[jr]
        if s["draft_probs"] is None:
            take[jr] = u[jr, 0].double() < px
            rest[torch.arange(jr.numel(), device="cuda"), x] = 0.0
        else:
            q = s["draft_probs"][d[judges]].double()
            take[jr] = u[jr, 0].double() * q[torch.arange(jr.numel(), device="cuda"), x] < px
            rest = rest.sub_(q).clamp_(min=0.0)
        p[jr] = torch.where(rest.sum(1, keepdim=True) > 0, rest, p[jr])
    drawn = _pick(p, u[:, 1])
    # a sequence's accepted drafts are those before its first row that does not accept
    first = torch.full((seqs,), rows, device="cuda").scatter_reduce_(0, of, torch.where(take, rows, r), "amin")
    accepted = first - (ends - (cu[1:] - cu[:-1]) - 1)
    ids = torch.where(r < first[of], torch.cat((drafts, drafts.new_zeros(1)))[torch.where(judges, d, drafts.numel())],
                      torch.where(r == first[of], drawn, -1))
    return {"ids": ids, "accepted": accepted.to(torch.int32)}


def _plain_attention(s):
    c, q, pool, table, length = s["case"], s["q"], s["pool"], s["table"].long(), s["length"].long()
    kv, dim, page = c["kv_heads"], c["head_dim"], c["page"]
    group = c["q_heads"] // kv
    cu = s["cu_new"].long()
    t = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[b]
    n, seqs, keys = s["max_new"], table.shape[0], table.shape[1] * page
    at = torch.arange(keys, device="cuda")
    held = (at[None] < length[:, None])[:, None, :, None]  # [seqs, 1, keys, 1]

    def side(which):  # [seqs, kv, keys, dim]; what lies behind a sequence's end counts as zero
        x = pool[:, 0, which][table.clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(seqs, kv, keys, dim)
        return torch.where(held, x.float(), 0.0)

    qp = torch.zeros((seqs, n, kv, group, dim), dtype=torch.float32, device="cuda")
    qp[b, i] = q.float().view(-1, kv, group, dim)
    qp = qp.permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * n, dim)
    scores = torch.matmul(qp, side(0).transpose(2, 3)).mul_(1.0 / math.sqrt(dim)).view(seqs, kv, group, n, keys)
    p = (length - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device="cuda")[None]  # position of each query
    seen = (at[None, None] < length[:, None, None]) & ((at[None, None] > p[:, :, None] - c["window"]) | (at[None, None] < c["sinks"]))
    if c["causal"]:
        seen &= at[None, None] <= p[:, :, None]
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    weight = scores.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.view(seqs, kv, group * n, keys), side(1)).view(seqs, kv, group, n, dim)
    out = out / torch.where(total == 0.0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4)[b, i].reshape(q.shape).to(q.dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2)[b, i].reshape(q.shape[:2])}


_plain = {"sample": _plain_sample, "verify": _plain_verify, "attention": _plain_attention}
_own = {"sample": _own_sample, "verify": _own_verify, "attention": _own_attention}


# ---- the definitions in 64 bits -----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "verify": _exact_verify, "attention": _exact_attention}[case["op"]](case, s)


def _exact_row(x, t, k, p, m):
    """The probabilities of one row's tokens, from the distinct logits and how often each occurs."""
    x = x.double()
    value, count = torch.unique(x[torch.isfinite(x)], return_counts=True)
    if value.numel() == 0:
        return torch.zeros_like(x)
    value, count = value.flip(0), count.flip(0)
    if t <= 0:
        prob = torch.zeros_like(x)
        prob[torch.nonzero(x == value[0])[0, 0]] = 1.0
        return prob
    weight = torch.exp((value - value[0]) / t)
    before = torch.cumsum(count, 0) - count  # tokens of larger logits
    keep = count.clone()  # of each logit, the first so many tokens stay
    if k > 0:
        keep = torch.minimum(keep, (k - before).clamp(min=0))
    if p < 1:
        mass = weight * keep
        left = p * mass.sum() - (torch.cumsum(mass, 0) - mass)  # of the nucleus, before each logit
        keep = torch.minimum(keep, torch.ceil(left / weight.clamp(min=1e-300)).clamp(min=0, max=x.numel()).long())
        keep[0] = max(1, int(keep[0]))
    if m > 0:
        keep = torch.where(weight >= m, keep, 0)
    last = int(torch.nonzero(keep)[-1])
    prob = torch.where(x >= value[last], torch.exp((x - value[0]) / t), 0.0)
    ties = torch.nonzero(x == value[last])[:, 0]
    prob[ties[int(keep[last]):]] = 0.0
    return prob / prob.sum()


def _exact_rows(case, s):
    """(probabilities, its settings' index) of each row, in order."""
    names = ("temperature", "top_k", "top_p", "min_p")
    settings = list(zip(*[s["settings"][n].tolist() for n in names]))
    of = range(case["rows"]) if case["op"] == "sample" else [i for i, d in enumerate(_drafts(case)) for _ in range(d + 1)]
    for row, i in enumerate(of):
        yield _exact_row(s["logits"][row], *settings[i])


def _exact_pick(prob, u):
    if float(prob.sum()) <= 0:
        return -1
    upto = torch.cumsum(prob, 0)
    return int(torch.searchsorted(upto, (u.double() * upto[-1]).reshape(1), right=True))


def _exact_sample(case, s):
    ids, probs = [], []
    for prob, u in zip(_exact_rows(case, s), s["uniforms"]):
        ids.append(_exact_pick(prob, u))
        if case["probs"]:
            probs.append(prob)
    ids = torch.tensor(ids, device="cuda")
    return {"ids": ids, "probs": torch.stack(probs)} if case["probs"] else {"ids": ids}


def _exact_verify(case, s):
    ids, accepted, row, draft = [], [], 0, 0
    rows = _exact_rows(case, s)
    for n in _drafts(case):
        taken, out = 0, []
        for i in range(n + 1):
            prob, u = next(rows), s["uniforms"][row + i]
            if len(out) > taken:
                out.append(-1)  # behind the token that ended the sequence's cycle
                continue
            if i < n:
                x = int(s["drafts"][draft + i])
                q = None if s["draft_probs"] is None else s["draft_probs"][draft + i].double()
                if float(u[0].double() * (1.0 if q is None else q[x])) < float(prob[x]):
                    taken += 1
                    out.append(x)
                    continue
                rest = torch.clamp(prob - q, min=0.0) if q is not None else prob.clone().index_fill_(0, s["drafts"][draft + i][None], 0.0)
                prob = rest if float(rest.sum()) > 0 else prob
            out.append(_exact_pick(prob, u[1]))
        ids += out
        accepted.append(taken)
        row, draft = row + n + 1, draft + n
    return {"ids": torch.tensor(ids, device="cuda"), "accepted": torch.tensor(accepted, dtype=torch.int32, device="cuda")}


def _exact_attention(case, s):
    new, ctx = _lengths(case)
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pages = s["table"][b, : -(-(n + c) // case["page"])].long()
        tokens = s["pool"][pages, 0].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, : n + c]  # [2, heads, tokens, dim]
        key = torch.arange(n + c, device="cuda")
        query = torch.arange(c, c + n, device="cuda")[:, None]
        hidden = (key <= query - case["window"]) & (key >= case["sinks"])
        if case["causal"]:
            hidden |= key > query
        for h in range(case["q_heads"]):
            k, v = tokens[0, h // group].double(), tokens[1, h // group].double()
            score = (s["q"][t : t + n, h].double() @ k.T) / math.sqrt(case["head_dim"])
            score = score.masked_fill_(hidden, float("-inf"))
            lse[t : t + n, h] = torch.logsumexp(score, 1)
            out[t : t + n, h] = torch.softmax(score, 1) @ v
        t += n
    return {"out": out, "lse": lse}
