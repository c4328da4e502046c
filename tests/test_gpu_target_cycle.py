"""The target's calls together, as examples/target_cycle.py runs them: the
draft-verify loop over the paged cache emits what the target alone would."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def _prompt(ex, target):
    g = torch.Generator().manual_seed(1)
    prompt = torch.randint(0, target.V, (target.B, 40), generator=g,
                           dtype=torch.int32).cuda()
    lengths = torch.tensor([40, 17, 1, 33], dtype=torch.int32, device="cuda")
    return prompt, lengths


def test_greedy_loop_equals_decoding_token_by_token(lib):
    """T = 0: the loop's tokens are the target's own greedy tokens, decoded
    one at a time over a cache of its own."""
    import target_cycle as ex
    target = ex.ToyTarget(4, 4)
    prompt, lengths = _prompt(ex, target)
    tokens, length, stats = ex.generate(target, prompt, lengths, 12,
                                        ex.Filters(T=0.0))
    assert int(stats[1]) == 4 * 12
    assert int(stats[2]) == int((length - 1).sum())
    alone = ex.ToyTarget(4, 4)
    l = alone.logits(prompt, torch.zeros_like(lengths), lengths)
    last = l[torch.arange(4), lengths.long() - 1].argmax(1).to(torch.int32)
    for i in range(int(length.max())):
        live = i < length
        assert torch.equal(tokens[live, i], last[live]), i
        l = alone.logits(last[:, None].contiguous(), lengths + i)
        last = l[:, 0].argmax(1).to(torch.int32)
    lib.dflash_check()


def test_filtered_loop_emits_only_kept_tokens(lib):
    """With top-k = 3 every emitted token is among the three largest logits
    of its position, recomputed over a cache of its own."""
    import target_cycle as ex
    target = ex.ToyTarget(4, 4)
    prompt, lengths = _prompt(ex, target)
    tokens, length, _ = ex.generate(target, prompt, lengths, 8,
                                    ex.Filters(T=1.3, top_k=3))
    n = int(length.min())
    alone = ex.ToyTarget(4, 4)
    alone.logits(prompt, torch.zeros_like(lengths), lengths)
    l = alone.logits(tokens[:, :n].contiguous(), lengths)
    for i in range(1, n):
        top = l[:, i - 1].topk(4, dim=1)
        near = (top.values[:, 2] - top.values[:, 3]) < 0.05  # caches differ
        k = torch.where(near, 4, 3)[:, None]
        allowed = torch.where(torch.arange(4, device="cuda") < k,
                              top.indices, -1)
        assert (allowed == tokens[:, i, None]).any(1).all(), i
    lib.dflash_check()


def test_example_runs(lib, capsys):
    import target_cycle as ex
    ex.main()
    assert capsys.readouterr().out.count("verification passes") == 2
