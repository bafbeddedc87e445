"""The example that runs the layer operators together: it learns, and its prompt and single-step paths give what its
training path gives."""
import os
import sys

import pytest
import torch

from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_learns(gpu):
    import recurrent_lm as lm
    say("example training")
    losses = lm.train(lm.Model(), 100, log=lambda s: None)
    # log(32) = 3.47 knows nothing
    assert losses[-1] < 1.5 < 3.4 < losses[0], (losses[0], losses[-1])


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_and_steps_agree_with_the_whole_sequence(gpu, fp8):
    """fp32 throughout: the paths differ in the order of sums only, a few hundred roundings of 2^-24 of logits of order
    one; with the norms in 8 bits each is within 2^-4 of itself, and the logits move by less than half of their size."""
    import recurrent_lm as lm
    say(f"example generation fp8={fp8}")
    model = lm.Model(seed=3)
    tokens = lm.phrases(3, 50, 8, 32, torch.Generator().manual_seed(5))
    lengths = torch.tensor([30, 1, 17], dtype=torch.int32, device=gpu)
    with torch.no_grad():
        whole = model(tokens)
    got, states = model.prompt(tokens[:, :30], lengths, fp8)
    slots = torch.tensor([2, 0, 4], dtype=torch.int32, device=gpu)
    cache = []
    for S in states:
        c = S.new_zeros(5, *S.shape[1:])
        c[slots.long()] = S
        cache.append(c)
    size = float(whole.abs().max())
    tol = 0.5 * size if fp8 else 1e-3 * size
    for n in range(15):
        for b in range(3):
            want = whole[b, int(lengths[b]) - 1 + n]
            assert float((got[b] - want).abs().max()) <= tol, (n, b)
        now, before = (torch.stack([tokens[b, int(lengths[b]) + n - j] for b in range(3)]) for j in (0, 1))
        got = model.step(now, before, cache, slots, fp8)
