"""The key-value side of a draft or verify step, measured: rotary positions written into a paged
cache, attention of a chunk of new tokens over that cache, and the cache's page operations.

Each case is one call (or the two calls that belong together) as a serving or training loop
makes them.  ``own`` selects the library's kernels; otherwise ``run`` computes the same thing
from elementary torch operations in 32 bits, rounded once at the end.

The cache of all cases: pool [pages, layers, 2 (k, v), kv heads, page size, head dim], table
int32 [sequences, pages of a sequence] (-1 where there is none), length int32 [sequences], refs
int32 [pages] (0: free).  New pages are the lowest-numbered free ones.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TURN = 1 << 64  # one turn in the fixed-point frequencies


# ---- the cases ---------------------------------------------------------------------------
def listed():
    heads = dict(q_heads=32, kv_heads=8, head_dim=128)
    return [
        # one user's next token over a short conversation: launch latency is all of it
        dict(name="attention_one_token", op="attention", **heads, dtype="bf16", page=16, seqs=1, new_lo=1, new_hi=1,
             ctx_lo=776, ctx_hi=776, causal=True, window=0, salt=1),
        # a draft block of 7 positions for 16 ragged requests, every position seeing the whole block
        dict(name="attention_draft_block", op="attention", **heads, dtype="bf16", page=16, seqs=16, new_lo=7, new_hi=7,
             ctx_lo=300, ctx_hi=6000, causal=False, window=0, salt=2),
        # verifying 1 to 8 drafted tokens over long documents: the cache's bytes bound it
        dict(name="attention_verify_long", op="attention", **heads, dtype="fp16", page=64, seqs=8, new_lo=1, new_hi=8,
             ctx_lo=16000, ctx_hi=66000, causal=True, window=0, salt=3),
        # ragged prompt chunks of a small model with a sliding window, 7 query heads to a kv head
        dict(name="attention_window_chunks", op="attention", q_heads=28, kv_heads=4, head_dim=64, dtype="fp16", page=32,
             seqs=6, new_lo=90, new_hi=1500, ctx_lo=0, ctx_hi=2100, causal=True, window=1000, salt=4),
        # the second half of a long prompt: the tensor cores bound it
        dict(name="attention_prefill_long", op="attention", **heads, dtype="bf16", page=64, seqs=1, new_lo=8192,
             new_hi=8192, ctx_lo=8192, ctx_hi=8192, causal=True, window=0, salt=5),
        # rotating and appending one token for each of 24 requests
        dict(name="append_tokens", op="append", **heads, dtype="bf16", page=16, seqs=24, new_lo=1, new_hi=1, ctx_lo=20,
             ctx_hi=30000, rotary=128, layout="half", factor=4.0, amplitude=1.0, salt=6),
        # the prompts of five new requests, half of each head rotated, scaled for a long context
        dict(name="append_prompts", op="append", **heads, dtype="bf16", page=64, seqs=5, new_lo=500, new_hi=4000,
             ctx_lo=0, ctx_hi=9000, rotary=64, layout="half", factor=8.0, amplitude=1.2079, salt=7),
        # a training step's rotation with its gradient, interleaved pairs
        dict(name="rotary_training", op="rotary", heads=40, head_dim=128, dtype="bf16", tokens=8190, rotary=128,
             layout="interleaved", factor=1.0, amplitude=1.0, salt=8),
        # beam search: four beams of one prompt reordered, five layers
        dict(name="fork_beams", op="fork", kv_heads=8, head_dim=128, dtype="bf16", page=16, layers=5, groups=1, width=4,
             ring=True, ctx_lo=700, ctx_hi=700, salt=9),
        # 32 samples from each of eight prompts, the cache of 36 layers: the page copies' bytes bound it
        dict(name="fork_samples", op="fork", kv_heads=8, head_dim=128, dtype="bf16", page=16, layers=36, groups=8,
             width=33, ring=False, ctx_lo=300, ctx_hi=1500, salt=10),
        # a bounded cache: 16 requests take 32 tokens each and drop as many from behind their first 4
        dict(name="compact_window", op="compact", kv_heads=8, head_dim=128, dtype="bf16", page=16, layers=4, seqs=16,
             sinks=4, drop=32, scattered=False, ctx_lo=900, ctx_hi=4100, salt=11),
        # 64 requests end and 64 others are admitted in their place: page bookkeeping alone
        dict(name="admit_requests", op="admit", kv_heads=2, head_dim=64, dtype="bf16", page=16, layers=1, seqs=64,
             ctx_lo=60, ctx_hi=8000, salt=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "rotary", "fork", "compact", "admit"])
    salt = rng.randrange(1, 1 << 30)
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    if op == "attention":
        group = rng.choice([1, 2, 3, 4, 6, 7, 8])
        seqs = _log(rng, 1, 48)
        new = rng.choice([1, _log(rng, 1, 16), _log(rng, 16, 6000)])
        ctx = _log(rng, 1, 60000)
        while seqs > 1 and seqs * new * (new + ctx) * kv * group * dim > 4e11 or seqs * (ctx + new) * kv * dim > 3e8:
            seqs, ctx = max(1, seqs // 2), max(1, ctx // 2)
        while new * (new + ctx) * kv * group * dim > 4e11:
            new = max(1, new // 2)
        return dict(op=op, q_heads=kv * group, kv_heads=kv, head_dim=dim, dtype=dtype, page=page, seqs=seqs,
                    new_lo=max(1, new // rng.choice([1, 1, 3])), new_hi=new, ctx_lo=rng.choice([0, ctx // 3, ctx]), ctx_hi=ctx,
                    causal=rng.random() < 0.75, window=rng.choice([0, 0, _log(rng, 5, 5000)]), salt=salt)
    rotary = rng.choice([dim, dim // 2, dim // 4])
    layout = rng.choice(["half", "interleaved"])
    factor = rng.choice([1.0, 4.0, 8.0])
    amplitude = rng.choice([1.0, 0.1 * math.log(factor) + 1.0])
    if op == "append":
        seqs = _log(rng, 1, 100)
        new = rng.choice([1, _log(rng, 1, max(2, 12000 // seqs))])
        return dict(op=op, q_heads=kv * rng.choice([1, 3, 4, 8]), kv_heads=kv, head_dim=dim, dtype=dtype, page=page,
                    seqs=seqs, new_lo=max(1, new // 4), new_hi=new, ctx_lo=0, ctx_hi=_log(rng, 1, 40000), rotary=rotary,
                    layout=layout, factor=factor, amplitude=amplitude, salt=salt)
    if op == "rotary":
        return dict(op=op, heads=_log(rng, 1, 48), head_dim=dim, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    tokens=_log(rng, 1, 8000), rotary=rotary, layout=layout, factor=factor, amplitude=amplitude, salt=salt)
    if op == "fork":
        ring = rng.random() < 0.5
        groups, width = _log(rng, 1, 8), _log(rng, 2, 24)
        return dict(op=op, kv_heads=kv, head_dim=dim, dtype=dtype, page=rng.choice([16, 32]), layers=_log(rng, 1, 24),
                    groups=groups, width=width, ring=ring, ctx_lo=1, ctx_hi=_log(rng, 40, 1500), salt=salt)
    if op == "compact":
        ctx = _log(rng, 100, 4000)
        return dict(op=op, kv_heads=kv, head_dim=dim, dtype=dtype, page=rng.choice([16, 32, 64]), layers=_log(rng, 1, 4),
                    seqs=_log(rng, 1, 16), sinks=rng.choice([0, 1, 4, 33]), drop=_log(rng, 1, 64),
                    scattered=rng.random() < 0.5, ctx_lo=ctx // 2 + 1, ctx_hi=ctx, salt=salt)
    return dict(op=op, kv_heads=kv, head_dim=dim, dtype=dtype, page=rng.choice([16, 32, 64]), layers=1,
                seqs=_log(rng, 1, 100), ctx_lo=1, ctx_hi=_log(rng, 50, 8000), salt=salt)


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
    return _spread(case, case.get("new_lo", 0), case.get("new_hi", 0), n, "new"), _spread(
        case, case["ctx_lo"], case["ctx_hi"], n, "ctx")


def _fork_rows(case):
    """(tokens of each row, source rows, target rows): rows of one group are next to each other."""
    g, w = case["groups"], case["width"]
    tokens = _spread(case, case["ctx_lo"], case["ctx_hi"], g, "fork")
    if case["ring"]:  # every beam continues the next one of its group
        dst = list(range(g * w))
        src = [i // w * w + (i + 1) % w for i in dst]
    else:  # every row of a group is a new sample of its first
        dst = [i for i in range(g * w) if i % w]
        src = [i // w * w for i in dst]
    return [tokens[i // w] for i in range(g * w)], src, dst


def _frequencies(case):
    """Turns of each pair of a head for one position, as a 64-bit fraction of a turn.  A factor other
    than 1 divides the slow pairs' by it, keeps the fast pairs' (32 turns and more within the
    4096 positions trained on) and goes evenly between."""
    half = case["rotary"] // 2
    turns = [10000.0 ** (-j / half) / (2.0 * math.pi) for j in range(half)]
    keep = [min(1.0, max(0.0, (4096.0 * f - 1.0) / 31.0)) for f in turns]
    turns = [f * (k + (1.0 - k) / case["factor"]) for f, k in zip(turns, keep)]
    whole = [int(round(f * TURN)) % TURN for f in turns]
    return turns, [w - TURN if w >= TURN // 2 else w for w in whole]


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "attention":
        new, ctx = _lengths(case)
        pairs = keys = 0
        for n, c in zip(new, ctx):
            length = n + c
            lo = [max(0, c + i - case["window"] + 1) if case["window"] else 0 for i in range(n)]
            hi = [c + i + 1 if case["causal"] else length for i in range(n)]
            pairs += sum(h - x for h, x in zip(hi, lo))
            keys += length - lo[0]
        row = case["head_dim"] * size
        rows = sum(new) * case["q_heads"]
        return {"bytes": 2 * rows * row + rows * 4 + 2 * keys * case["kv_heads"] * row,
                "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}
    if op == "append":
        tokens = sum(_lengths(case)[0])
        heads = case["q_heads"] + 2 * case["kv_heads"]
        turned = tokens * (case["q_heads"] + case["kv_heads"]) * case["rotary"]
        return {"bytes": 2 * tokens * heads * case["head_dim"] * size, "flops": 3 * turned}
    if op == "rotary":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["head_dim"] * size + 4 * case["tokens"], "flops": 6 * n * case["rotary"]}
    token = case["layers"] * 2 * case["kv_heads"] * case["head_dim"] * size
    if op == "fork":
        tokens, src, dst = _fork_rows(case)
        pages = sum(-(-tokens[d] // case["page"]) for d in dst)
        return {"bytes": 2 * token * sum(tokens[d] % case["page"] for d in dst) + 12 * pages, "flops": 0}
    if op == "compact":
        _, ctx = _lengths(case)
        return {"bytes": sum(2 * token * (c - case["sinks"]) + 4 * (c - case["sinks"]) for c in ctx), "flops": 0}
    _, ctx = _lengths(case)
    return {"bytes": sum(24 * -(-c // case["page"]) for c in ctx), "flops": 0}


# ---- inputs -------------------------------------------------------------------------------
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _cache(case, gen, layers, tokens, lead=None, spare=0, room=0):
    """A cache whose rows hold `tokens`, on pages scattered over the pool as in a server that has run
    for a while.  Row i shares the full pages of row lead[i] (none where that is i itself); every
    row has room for `room` more tokens in its table."""
    page, dtype = case["page"], TYPES[case["dtype"]]
    wide = max(1, max(-(-(t + room) // page) for t in tokens))
    table, used = [], 0
    for i, t in enumerate(tokens):
        full = t // page if lead is not None and lead[i] != i else 0
        own_pages = -(-t // page) - full
        row = (table[lead[i]][:full] if full else []) + list(range(used, used + own_pages))
        table.append(row + [-1] * (wide - len(row)))
        used += own_pages
    pages = used + spare + 3
    pool = torch.randn((pages, layers, 2, case["kv_heads"], page, case["head_dim"]), generator=gen, device="cuda", dtype=dtype)
    order = torch.cat((torch.randperm(pages, generator=gen, device="cuda"), torch.full((1,), -1, device="cuda")))
    table = order[torch.tensor(table, device="cuda")]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    held = table[table >= 0]
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    return {"pool": pool, "table": table.to(torch.int32), "refs": refs,
            "length": torch.tensor(tokens, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + case["salt"])
    s = {"case": case}
    op, dtype = case["op"], TYPES[case["dtype"]]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if op == "rotary":
        shape = (case["tokens"], case["heads"], case["head_dim"])
        s["x"], s["dy"] = _normal(gen, shape, dtype), _normal(gen, shape, dtype)
        s["positions"] = torch.randint(0, 32768, (case["tokens"],), generator=gen, device="cuda", dtype=torch.int32)
    elif op in ("attention", "append"):
        new, ctx = _lengths(case)
        s.update(_cache(case, gen, 1, [n + c for n, c in zip(new, ctx)]))
        s["max_new"] = max(new)
        s["cu_new"] = ints([sum(new[:i]) for i in range(len(new) + 1)])
        s["q"] = _normal(gen, (sum(new), case["q_heads"], case["head_dim"]), dtype)
        if op == "append":
            s["k"] = _normal(gen, (sum(new), case["kv_heads"], case["head_dim"]), dtype)
            s["v"] = _normal(gen, (sum(new), case["kv_heads"], case["head_dim"]), dtype)
        else:
            s["scale"] = 1.0 / math.sqrt(case["head_dim"])
    elif op == "fork":
        tokens, src, dst = _fork_rows(case)
        width = case["width"]
        if not case["ring"]:
            tokens = [0 if i % width else t for i, t in enumerate(tokens)]
        s.update(_cache(case, gen, case["layers"], tokens, [i // width * width for i in range(len(tokens))], spare=2 * len(dst)))
        s["src"], s["dst"] = ints(src), ints(dst)
    elif op == "compact":
        _, ctx = _lengths(case)
        sinks, drop = case["sinks"], case["drop"]
        s.update(_cache(case, gen, case["layers"], ctx, spare=len(ctx) * (2 + drop // case["page"]), room=drop))
        wide = max(ctx) - sinks
        at = torch.arange(wide, device="cuda")[None].expand(len(ctx), wide)
        count = ints(ctx)[:, None] - sinks
        if case["scattered"]:  # the kept tokens are spread over all that the row then has
            total = count + drop
            noise = torch.rand((len(ctx), wide + drop), generator=gen, device="cuda")
            noise = torch.where(torch.arange(wide + drop, device="cuda")[None] < total, noise, 2.0)
            chosen = torch.argsort(noise, dim=1)[:, :wide]
            chosen = torch.where(at < count, chosen, wide + drop)
            kept = torch.sort(chosen, dim=1).values + sinks
        else:
            kept = at + sinks + drop
        s["kept"] = torch.where(at < count, kept, 0).to(torch.int32).contiguous()
        s["n_kept"] = count[:, 0].contiguous()
        s["start"] = torch.full_like(s["n_kept"], sinks)
        s["add"] = torch.full_like(s["n_kept"], drop)
        s["rows"] = torch.arange(len(ctx), dtype=torch.int32, device="cuda")
    elif op == "admit":
        _, ctx = _lengths(case)
        s.update(_cache(case, gen, case["layers"], ctx, spare=5 * len(ctx)))
        s["rows"] = torch.randperm(len(ctx), generator=gen, device="cuda").to(torch.int32)
        s["add"] = ints(ctx)[s["rows"].long()].contiguous()
    if "rotary" in case:
        s["turns"] = torch.tensor(_frequencies(case)[1], dtype=torch.int64, device="cuda")
    if own:  # the cache and the frequencies as a program keeps them
        from dspark_draft_sampling_gb300 import api

        if "pool" in s:
            s["cache"] = api.PagedCache(s["pool"], s["table"], s["length"], s["refs"])
        if "rotary" in case:
            s["table_of"] = api.RotaryTable(s["turns"], layout=case["layout"], amplitude=case["amplitude"])
    return s


# ---- one pass -----------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    return (_own if own else _plain)[op](s)


def _own_attention(s):
    from dspark_draft_sampling_gb300 import api

    c = s["case"]
    out, lse = api.paged_attention(s["q"], s["cache"], 0, s["cu_new"], max_new=s["max_new"], causal=c["causal"],
                                   window=c["window"], scale=s["scale"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_append(s):
    from dspark_draft_sampling_gb300 import api

    q = api.rotary_append(s["q"], s["k"], s["v"], s["cache"], 0, s["cu_new"], s["table_of"])
    return {"q": q, "pool": s["pool"]}


def _own_rotary(s):
    from dspark_draft_sampling_gb300 import api

    return {"y": api.rotary(s["x"], s["positions"], s["table_of"]),
            "dx": api.rotary(s["dy"], s["positions"], s["table_of"], backward=True)}


def _books(s):
    return {"table": s["table"], "length": s["length"], "refs": s["refs"]}


def _own_fork(s):
    s["cache"].fork(s["src"], s["dst"])
    return {"pool": s["pool"], **_books(s)}


def _own_compact(s):
    s["cache"].extend(s["rows"], s["add"])
    s["cache"].compact(s["rows"], s["start"], s["kept"], s["n_kept"])
    return {"pool": s["pool"], **_books(s)}


def _own_admit(s):
    s["cache"].free(s["rows"])
    s["cache"].extend(s["rows"], s["add"])
    return _books(s)


# ---- the plain forms ----------------------------------------------------------------------
def _chunk(s):
    """Of every new token: its sequence, its place in the chunk and its position in the cache."""
    cu, length = s["cu_new"].long(), s["length"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[b]
    return b, i, length[b] - (cu[b + 1] - cu[b]) + i


def _plain_attention(s):
    c, q, pool, table, length = s["case"], s["q"], s["pool"], s["table"].long(), s["length"].long()
    kv, dim, page = c["kv_heads"], c["head_dim"], c["page"]
    group = c["q_heads"] // kv
    b, i, pos = _chunk(s)
    n, seqs, keys = s["max_new"], table.shape[0], table.shape[1] * page
    at = torch.arange(keys, device="cuda")
    held = (at[None] < length[:, None])[:, None, :, None]  # [seqs, 1, keys, 1]

    def side(which):  # [seqs, kv, keys, dim]; what lies behind a sequence's end counts as zero
        x = pool[:, 0, which][table.clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(seqs, kv, keys, dim)
        return torch.where(held, x.float(), 0.0)

    qp = torch.zeros((seqs, n, kv, group, dim), dtype=torch.float32, device="cuda")
    qp[b, i] = q.float().view(-1, kv, group, dim)
    qp = qp.permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * n, dim)
    scores = torch.matmul(qp, side(0).transpose(2, 3)).mul_(s["scale"]).view(seqs, kv, group, n, keys)
    cu = s["cu_new"].long()
    p = (length - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device="cuda")[None]  # position of each query
    seen = (at[None, None] < length[:, None, None]).expand(seqs, n, keys)
    if c["causal"]:
        seen = seen & (at[None, None] <= p[:, :, None])
    if c["window"]:
        seen = seen & (at[None, None] > p[:, :, None] - c["window"])
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


def _turned(s, x, positions, sign):
    """The rotation of x [tokens, heads, dim], in 32 bits; the angle's whole turns fall off in 64-bit
    fixed point, so a long context costs no precision."""
    c = s["case"]
    half = c["rotary"] // 2
    part = positions.long()[:, None] * s["turns"][None]  # modulo one turn
    angle = (part >> 32).float() * (2.0 * math.pi / 2.0**32)
    cos, sin = (c["amplitude"] * angle.cos())[:, None], (sign * c["amplitude"] * angle.sin())[:, None]
    y = x.float()
    r, rest = y[..., : c["rotary"]], y[..., c["rotary"]:]
    if c["layout"] == "half":
        a, b = r[..., :half], r[..., half:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r, rest), -1).to(x.dtype)


def _plain_append(s):
    b, _, pos = _chunk(s)
    page = s["case"]["page"]
    to = s["table"].long()[b, pos // page]
    rows = s["pool"].permute(0, 4, 1, 2, 3, 5)  # [pages, slots, layers, 2, heads, dim]
    rows[to, pos % page, 0, 0] = _turned(s, s["k"], pos, 1.0)
    rows[to, pos % page, 0, 1] = s["v"]
    return {"q": _turned(s, s["q"], pos, 1.0), "pool": s["pool"]}


def _plain_rotary(s):
    return {"y": _turned(s, s["x"], s["positions"], 1.0), "dx": _turned(s, s["dy"], s["positions"], -1.0)}


def _fresh(refs, wanted):
    """For every true entry of `wanted`, in order, the next lowest-numbered free page."""
    rank = torch.cumsum((refs == 0).long(), 0)
    order = torch.cumsum(wanted.reshape(-1).long(), 0).reshape(wanted.shape)
    return torch.searchsorted(rank, order).clamp(max=refs.numel() - 1).to(torch.int32)


def _count(refs, pages, mask, by):
    refs.index_add_(0, pages[mask].long(), torch.full_like(pages[mask], by))


def _plain_extend(s, rows, add):
    page, table, length, refs = s["case"]["page"], s["table"], s["length"], s["refs"]
    slot = torch.arange(table.shape[1], device="cuda")[None]
    old = length[rows]
    new = old + add
    wanted = (slot * page >= old[:, None]) & (slot * page < new[:, None])
    fresh = _fresh(refs, wanted)
    table[rows] = torch.where(wanted, fresh, table[rows])
    _count(refs, fresh, wanted, 1)
    length[rows] = new


def _plain_fork(s):
    page, table, length, refs = s["case"]["page"], s["table"], s["length"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    slot = torch.arange(table.shape[1], device="cuda")[None]
    was, tokens, old = table[src], length[src], table[dst]
    moves = (src != dst)[:, None]
    last = (slot == (tokens // page)[:, None]) & (tokens % page != 0)[:, None] & moves
    fresh = _fresh(refs, last)
    now = torch.where(last, fresh, was)
    _count(refs, old, (old >= 0) & moves, -1)
    _count(refs, now, (now >= 0) & moves, 1)
    f = torch.arange(page, device="cuda")[None] < (tokens % page)[:, None]
    f = f & last.any(1, keepdim=True)
    which, filled = f.nonzero(as_tuple=True)
    lastpage = (tokens // page).long()[which]
    rows = s["pool"].permute(0, 4, 1, 2, 3, 5)
    rows[now[which, lastpage].long(), filled] = rows[was[which, lastpage].long(), filled]
    table[dst] = torch.where(moves, now, old)
    length[dst] = tokens
    return {"pool": s["pool"], **_books(s)}


def _plain_compact(s):
    _plain_extend(s, s["rows"].long(), s["add"])
    page, table, length, refs = s["case"]["page"], s["table"], s["length"], s["refs"]
    r, start, kept, count = s["rows"].long(), s["start"].long(), s["kept"].long(), s["n_kept"].long()
    new = start + count
    slot = torch.arange(table.shape[1], device="cuda")[None]
    was = table[r]
    stays = slot * page < new[:, None]
    touched = stays & (slot >= (start // page)[:, None])
    shared = touched & (refs[was.clamp(min=0).long()] > 1)
    now = torch.where(shared, _fresh(refs, shared), torch.where(stays, was, -1))
    # the tokens of every touched page: those before `start` where they are, the kept ones moved up
    first = start // page * page
    j = first[:, None] + torch.arange(int((new - first).max()), device="cuda")[None]
    k = j - start[:, None]
    source = torch.where(k < 0, j, kept.gather(1, k.clamp(min=0, max=kept.shape[1] - 1)))
    which, at = (j < new[:, None]).nonzero(as_tuple=True)
    j, source = j[which, at], source[which, at]
    rows = s["pool"].permute(0, 4, 1, 2, 3, 5)
    rows[now[which, j // page].long(), j % page] = rows[was[which, source // page].long(), source % page]
    _count(refs, was, (was >= 0) & (shared | ~stays), -1)
    _count(refs, now, shared, 1)
    table[r] = now
    length[r] = new.to(torch.int32)
    return {"pool": s["pool"], **_books(s)}


def _plain_admit(s):
    table, length, refs, rows = s["table"], s["length"], s["refs"], s["rows"].long()
    was = table[rows]
    _count(refs, was, was >= 0, -1)
    table[rows] = -1
    length[rows] = 0
    _plain_extend(s, rows, s["add"])
    return _books(s)


_plain = {"attention": _plain_attention, "append": _plain_append, "rotary": _plain_rotary, "fork": _plain_fork,
          "compact": _plain_compact, "admit": _plain_admit}
_own = {"attention": _own_attention, "append": _own_append, "rotary": _own_rotary, "fork": _own_fork,
        "compact": _own_compact, "admit": _own_admit}


# ---- the definitions in 64 bits -----------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op not in ("attention", "append", "rotary"):
        return None
    s = prepare(case, seed)
    if op == "attention":
        return _exact_attention(case, s)
    if op == "rotary":
        pos = s["positions"].tolist()
        return {"y": _exact_turn(case, s["x"], pos, 1), "dx": _exact_turn(case, s["dy"], pos, -1)}
    new, ctx = _lengths(case)
    pos = [c + i for n, c in zip(new, ctx) for i in range(n)]
    pool = s["pool"].double()
    k = _exact_turn(case, s["k"], pos, 1)
    t, pages = 0, s["table"].tolist()
    for b, (n, c) in enumerate(zip(new, ctx)):
        p = torch.arange(c, c + n, device="cuda")
        page = torch.tensor(pages[b], device="cuda")[p // case["page"]]
        pool[page, 0, 0, :, p % case["page"]] = k[t : t + n]
        pool[page, 0, 1, :, p % case["page"]] = s["v"][t : t + n].double()
        t += n
    return {"q": _exact_turn(case, s["q"], pos, 1), "pool": pool}


def _exact_turn(case, x, positions, sign):
    x = x.double()
    half = case["rotary"] // 2
    turns = torch.tensor(_frequencies(case)[0], dtype=torch.float64, device="cuda")
    angle = torch.tensor(positions, dtype=torch.float64, device="cuda")[:, None] * turns * (2.0 * math.pi)
    number = torch.polar(torch.full_like(angle, case["amplitude"]), sign * angle)[:, None]  # complex
    at = torch.arange(half, device="cuda")
    first, second = (at, at + half) if case["layout"] == "half" else (2 * at, 2 * at + 1)
    z = torch.complex(x[..., first], x[..., second]) * number
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


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
        hidden = torch.zeros((n, n + c), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= key > query
        if case["window"]:
            hidden |= key <= query - case["window"]
        for h in range(case["q_heads"]):
            k, v = tokens[0, h // group].double(), tokens[1, h // group].double()
            score = (s["q"][t : t + n, h].double() @ k.T) / math.sqrt(case["head_dim"])
            score = score.masked_fill_(hidden, float("-inf"))
            lse[t : t + n, h] = torch.logsumexp(score, 1)
            out[t : t + n, h] = torch.softmax(score, 1) @ v
        t += n
    return {"out": out, "lse": lse}
