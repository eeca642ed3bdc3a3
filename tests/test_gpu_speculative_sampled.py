"""The example's cycle with drawn tokens and a bounded view for the drafter: that it keeps what it says, and that its greedy form is what picking the
largest logits gives."""
import pytest
import torch

from dspark_draft_sampling_gb300 import api
from examples import speculative_cycle as example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,cycles,settings", [(3, 3, dict(temperature=0.8, top_p=0.9)), (9, 2, dict(temperature=1.3, window=16, sinks=4)),
                                               (2, 4, dict(window=20, sinks=2))])
def test_cycles_with_drawn_tokens(n, cycles, settings):
    cache, _, prompts, accepted = example.run(n, cycles, **settings)
    kept = torch.stack([k for _, k in accepted]).sum(0)
    assert cache.length[:n].tolist() == [len(p) + int(k) for p, k in zip(prompts, kept)]
    for (chunk, keep), (following, _) in zip(accepted, accepted[1:]):
        assert (keep >= 1).all() and (keep <= example.BLOCK).all()
        assert ((following[:, 0] >= 0) & (following[:, 0] < example.VOCAB)).all() and chunk.shape == following.shape


def test_the_greedy_cycle_is_what_the_largest_logits_give(monkeypatch):
    """Every call of verify_drafts at temperature 0 against the longest agreeing prefix of the drafts with the argmax."""
    seen = []

    def spy(logits, drafts, cu, uniforms, **kw):
        got = judge(logits, drafts, cu, uniforms, **kw)
        seen.append((logits.clone(), drafts.clone(), *got))
        return got

    judge = api.verify_drafts
    monkeypatch.setattr(api, "verify_drafts", spy)
    example.run(4, 3)
    for logits, drafts, ids, taken in seen:
        best = logits.argmax(-1).view(4, example.BLOCK)
        drafts = drafts.view(4, example.BLOCK - 1)
        agree = (best[:, :-1] == drafts).int().cumprod(1).sum(1)
        assert torch.equal(agree.int(), taken)
        for s in range(4):
            a = int(taken[s])
            row = ids.view(4, example.BLOCK)[s].tolist()
            assert row[:a] == drafts[s, :a].tolist() and row[a] == int(best[s, a]) and row[a + 1:] == [-1] * (example.BLOCK - 1 - a)
