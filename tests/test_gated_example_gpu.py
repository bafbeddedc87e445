"""The example that runs the token path's operators together: its gradients are those of the same model in torch in 64
bits, its prompt and single-step paths give what its training path gives, and it trains and draws."""
import os
import sys

import pytest
import torch

from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def loss64(params, tokens, reset, width, layers):
    """The example's loss from its parameters, in plain torch."""
    import gated_lm as lm
    p = {n: t for n, t in params}
    x = p["table"][tokens[:, :-1]] * width ** 0.5
    h = torch.zeros_like(x)

    def norm(v, w):
        return v * (v.square().mean(-1, keepdim=True) + lm.EPS).rsqrt() * w

    new = reset[:, :-1, None]
    for i in range(layers):
        h = h + x
        x, r, g, z = torch.split(norm(h, p[f"norms.{i}"]) @ p[f"project.{i}"], width, dim=-1)
        log_a = -lm.RATE * torch.nn.functional.softplus(p[f"lam.{i}"]) * torch.sigmoid(r)
        a = torch.exp(log_a).masked_fill(new, 0.0)
        b = torch.sqrt(-torch.expm1(2 * log_a)).masked_fill(new, 1.0) * torch.sigmoid(g) * x
        s, rows = torch.zeros_like(x[:, 0]), []
        for t in range(x.shape[1]):
            s = a[:, t] * s + b[:, t]
            rows.append(s)
        x = (torch.stack(rows, 1) * torch.nn.functional.silu(z)) @ p[f"back.{i}"]
    logits = norm(h + x, p[f"norms.{layers}"]) @ p["head"]
    target = tokens[:, 1:].masked_fill(reset[:, 1:], -100)
    return torch.nn.functional.cross_entropy(logits.flatten(0, 1), target.flatten())


def test_gradients(gpu):
    """fp32 against 64 bits: products of up to 512 terms, sums over 400 places and two layers of them: some thousands of
    2^-24 of each parameter's largest gradient."""
    import gated_lm as lm
    say("gated example gradients")
    model = lm.Model(width=48, seed=2)
    tokens, reset = lm.documents(5, 81, 32, torch.Generator().manual_seed(3))
    names = [n for n, _ in model.named_parameters()]
    got = torch.autograd.grad(lm.loss_of(model, tokens, reset), list(model.parameters()))
    exact = [p.detach().double().requires_grad_() for p in model.parameters()]
    want = torch.autograd.grad(loss64(list(zip(names, exact)), tokens, reset, 48, 2), exact)
    for n, x, y in zip(names, got, want):
        assert (x.double() - y).abs().max() <= 4000 * 2.0 ** -24 * y.abs().max(), n


def test_prompt_and_steps_agree_with_the_whole_sequence(gpu):
    """fp32 throughout: the paths differ in the order of sums only, a few hundred roundings of 2^-24 of logits of order
    one."""
    import gated_lm as lm
    say("gated example generation")
    model = lm.Model(seed=3)
    tokens, _ = lm.documents(3, 40, 32, torch.Generator().manual_seed(5))
    lengths = torch.tensor([20, 1, 17], dtype=torch.int32, device=gpu)
    with torch.no_grad():
        whole = model(tokens, torch.zeros_like(tokens, dtype=torch.bool))
    got, states = model.prompt(tokens[:, :20].contiguous(), lengths)
    slots = torch.tensor([2, 0, 4], dtype=torch.int32, device=gpu)
    cache = []
    for S in states:
        c = S.new_zeros(5, S.shape[1])
        c[slots.long()] = S
        cache.append(c)
    tol = 1e-3 * float(whole.abs().max())
    for n in range(15):
        for b in range(3):
            assert float((got[b] - whole[b, int(lengths[b]) - 1 + n]).abs().max()) <= tol, (n, b)
        got = model.step(torch.stack([tokens[b, int(lengths[b]) + n] for b in range(3)]), cache, slots)


def test_it_runs(gpu):
    import gated_lm as lm
    say("gated example run")
    model = lm.Model(width=64, dtype=torch.bfloat16)
    losses = lm.train(model, 3, batch=8, log=lambda s: None)
    assert all(0.0 < x < 100.0 for x in losses)
    tokens, _ = lm.documents(4, 30, 32, torch.Generator().manual_seed(7))
    lengths = torch.tensor([30, 1, 12, 29], dtype=torch.int32, device=gpu)
    text, logs = lm.generate(model, tokens, lengths, 5, torch.Generator(gpu).manual_seed(1), temperature=0.8, top_k=10)
    assert text.shape == (4, 5) and 0 <= int(text.min()) and int(text.max()) < 32 and (logs <= 0).all()
    again, _ = lm.generate(model, tokens, lengths, 5, torch.Generator(gpu).manual_seed(1), temperature=0.8, top_k=10)
    assert torch.equal(text, again)
