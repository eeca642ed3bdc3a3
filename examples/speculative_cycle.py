"""A speculative-decoding cycle's key-value side, on random weights: prompts into the cache, a draft block, the
verification of the drafts, and the cache cut back to what was accepted.

    python examples/speculative_cycle.py [--cycles 3] [--requests 4]

One attention layer stands for the model: q, k and v are the weight-stationary projections of the hidden rows, and
the drafts come from the Markov sampler over the layer's output.  Nothing here needs the host to know a length."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dspark_draft_sampling_gb300 import api  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB, RANK, BLOCK, PAGE = 1024, 8, 2, 64, 4096, 64, 7, 16


class Layer:
    """Projections of one attention layer in fp16, and its place in the cache."""

    def __init__(self, gen):
        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen) * cols ** -0.5).half().cuda()

        self.qkv = weight((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.out = weight(HIDDEN, Q_HEADS * DIM)
        self.head = weight(VOCAB, HIDDEN)
        self.embed = weight(VOCAB, HIDDEN)
        self.rotary = api.RotaryTable(api.rotary_frequencies(DIM, 10000.0, scaling="by_parts", factor=4.0, original=4096))

    def project(self, weight, x, **kw):
        """Rows of x in blocks of the matvec's 16."""
        return torch.cat([api.ws_matvec(weight, rows.contiguous(), **kw) for rows in x.split(16)])

    def forward(self, tokens, cache, cu_new, rows, max_new, causal):
        """Attention of the tokens' rows over the cache, which they are written into; returns the logits."""
        x = self.embed[tokens]
        qkv = self.project(self.qkv, x).view(-1, Q_HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1)
        q = api.rotary_append(q, k, v, cache, 0, cu_new, self.rotary, rows=rows)
        y = api.paged_attention(q, cache, 0, cu_new, rows=rows, max_new=max_new, causal=causal)
        x = x + self.project(self.out, y.reshape(-1, Q_HEADS * DIM))
        return self.project(self.head, x, out_fp32=True)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(n, cycles):
    """`cycles` cycles of n requests: the cache, the layer, the requests' prompts, and each cycle's verified tokens with how many of them
    were kept."""
    gen = torch.Generator().manual_seed(0)
    layer = Layer(gen)
    w1, w2 = ((torch.randn(VOCAB, RANK, generator=gen) * 0.2).to(torch.bfloat16).cuda() for _ in range(2))
    # a row holds its prompt and a block each cycle; a request has its row's pages, its draft row two or three of its own
    lens = [20 + 13 * i for i in range(n)]
    pages = [-(-(length + BLOCK * (cycles + 1)) // PAGE) for length in lens]
    cache = api.PagedCache.empty(sum(pages) + 3 * n, 2 * n, max(pages), layers=1, kv_heads=KV_HEADS, page_size=PAGE, head_dim=DIM,
                                 dtype=torch.float16)

    # the prompts of all requests in one ragged chunk
    rows, cu = ints(range(n)), ints([sum(lens[:i]) for i in range(n + 1)])
    cache.extend(rows, ints(lens))
    prompt = torch.randint(VOCAB, (sum(lens),), generator=gen).cuda()
    logits = layer.forward(prompt, cache, cu, rows, max(lens), causal=True)
    last = logits[cu[1:].long() - 1].argmax(-1)

    # a second row for each request: it shares the prompt's pages and takes the draft block, which sees itself whole
    drafts = ints(range(n, 2 * n))
    accepted = []
    for _ in range(cycles):
        cache.fork(rows, drafts)
        block_cu = ints(range(0, BLOCK * n + 1, BLOCK))
        cache.extend(drafts, ints([BLOCK] * n))
        block = last[:, None].expand(n, BLOCK).reshape(-1)
        base = layer.forward(block, cache, block_cu, drafts, BLOCK, causal=False).view(n, BLOCK, VOCAB)
        prev = last.clone()
        ids = torch.cat([api.markov_draft(base[i:i + 8].contiguous(), w1, w2, None, prev[i:i + 8]) for i in range(0, n, 8)])

        # the target reads the last token and the drafts in one causal chunk, and keeps the longest agreeing prefix
        chunk = torch.cat((last[:, None], ids[:, :-1]), 1)
        cache.extend(rows, ints([BLOCK] * n))
        verdict = layer.forward(chunk.reshape(-1), cache, block_cu, rows, BLOCK, causal=True).argmax(-1).view(n, BLOCK)
        agree = (verdict == ids).int().cumprod(1).sum(1)
        keep = (agree + 1).clamp(max=BLOCK)
        last = verdict.gather(1, (keep - 1).long()[:, None])[:, 0]
        cache.compact(rows, (cache.length[:n] - BLOCK + keep).int())
        accepted.append((chunk, keep))
    cache.free(drafts)
    if cache.status():
        raise SystemExit("the cache refused a call")
    return cache, layer, prompt.split(lens), accepted


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cycles", type=int, default=3)
    ap.add_argument("--requests", type=int, default=4)
    a = ap.parse_args(argv)
    cache, _, _, accepted = run(a.requests, a.cycles)
    print("tokens kept a cycle:", torch.stack([keep for _, keep in accepted], 1).tolist())
    print("cache lengths:", cache.length[:a.requests].tolist(), "pages in use:", int((cache.refs > 0).sum()))
    return cache


if __name__ == "__main__":
    main()
