"""A small recurrent language model on the layer operators: trained, then run token by token.

    python examples/recurrent_lm.py [--steps 300] [--fp8]

Each layer adds what came before to the residual stream and norms the sum (mgs_rmsnorm_fwd, _bwd), projects it to
queries, keys, values and decays, runs linear attention over the steps (mgs_linattn_fwd, _bwd) and projects back.
Training clips the gradients by their global norm (mgs_clip_norm).  Generation reads a prompt in one pass, keeps each
sequence's states in a cache, and goes on one token at a time (mgs_linattn_step); with --fp8 the norms ahead of the
projections hand over 8-bit values and scales (mgs_rmsnorm_fwd_fp8).

The data are synthetic: sequences that repeat a random phrase, so that after the first pass through the phrase every
token can be known from the state.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scan_linear_rnns_amd as mgs  # noqa: E402

EPS = 1e-6


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, scale):
        o, _, _ = mgs.mgs_linattn_fwd(q, k, v, g, scale=scale, want_state=False)
        ctx.save_for_backward(q, k, v, g)
        ctx.scale = scale
        return o

    @staticmethod
    def backward(ctx, do):
        dq, dk, dv, dg, _ = mgs.mgs_linattn_bwd(*ctx.saved_tensors, do, scale=ctx.scale)
        return dq, dk, dv, dg, None


class AddNorm(torch.autograd.Function):
    """(norm of x + residual, x + residual)"""

    @staticmethod
    def forward(ctx, x, residual, w):
        y, h, rstd = mgs.mgs_rmsnorm_fwd(x.contiguous(), w, residual, eps=EPS)
        ctx.save_for_backward(h, w, rstd)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, w, rstd = ctx.saved_tensors
        dx, dw = mgs.mgs_rmsnorm_bwd(dy.contiguous(), h, w, rstd, dh=dh.contiguous())
        return dx, dx, dw.to(w.dtype)


class Model(torch.nn.Module):
    def __init__(self, vocab=32, width=128, layers=2, heads=4, key=32, dtype=torch.float32, seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)
        self.heads, self.key, self.value = heads, key, width // heads
        self.sizes = [heads * key, heads * key, width, heads]   # q, k, v, decays

        def weight(*shape):
            w = torch.randn(*shape, generator=gen) / math.sqrt(shape[0])
            return torch.nn.Parameter(w.to(device="cuda", dtype=dtype))

        self.embed = weight(vocab, width)
        self.before = weight(vocab + 1, width)   # of the token before; the last row stands ahead of the first
        self.project = torch.nn.ParameterList([weight(width, sum(self.sizes)) for _ in range(layers)])
        self.back = torch.nn.ParameterList([weight(width, width) for _ in range(layers)])
        self.norms = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(width, device="cuda", dtype=dtype))
                                             for _ in range(layers + 1)])
        self.head = weight(width, vocab)
        # heads that forget over some 2 to 100 steps
        self.rate = torch.logspace(-2, -0.3, heads, device="cuda")

    def split(self, i, y):
        """Layer i's queries, keys, values (views of one projection) and log decays of normed inputs y (...,width)."""
        q, k, v, d = torch.split(y @ self.project[i], self.sizes, dim=-1)
        heads = (self.heads, -1)
        return q.unflatten(-1, heads), k.unflatten(-1, heads), v.unflatten(-1, heads), \
            -self.rate * torch.nn.functional.softplus(d.float())

    def inputs(self, tokens, previous):
        return self.embed[tokens] + self.before[previous]

    def shifted(self, tokens):
        return torch.cat([torch.full_like(tokens[:, :1], self.before.shape[0] - 1), tokens[:, :-1]], dim=1)

    def forward(self, tokens):
        x = self.inputs(tokens, self.shifted(tokens))
        h = torch.zeros_like(x)
        for i in range(len(self.project)):
            y, h = AddNorm.apply(x, h, self.norms[i])
            o = LinearAttention.apply(*self.split(i, y), self.key ** -0.5)
            x = o.flatten(2) @ self.back[i]
        y, _ = AddNorm.apply(x, h, self.norms[-1])
        return y @ self.head

    # ---- generation

    def normed(self, x, h, i, fp8):
        """The norm without a gradient; the residual stream h is updated in place."""
        if not fp8:
            return mgs.mgs_rmsnorm_fwd(x, self.norms[i], h, eps=EPS, h=h)[0]
        y8, scale, _ = mgs.mgs_rmsnorm_fwd_fp8(x, self.norms[i], h, eps=EPS, h=h)
        return (y8.float() * scale).to(x.dtype)   # where an 8-bit product would take both

    @torch.no_grad()
    def prompt(self, tokens, lengths, fp8=False):
        """Reads prompts of unlike lengths; logits after each one's last token, and the states."""
        B, T = tokens.shape
        x = self.inputs(tokens, self.shifted(tokens))
        h, states = torch.zeros_like(x), []
        for i in range(len(self.project)):
            o, S, _ = mgs.mgs_linattn_fwd(*self.split(i, self.normed(x, h, i, fp8)), lengths=lengths,
                                          scale=self.key ** -0.5)
            states.append(S)
            x = o.flatten(2) @ self.back[i]
        last = (torch.arange(B, device="cuda"), lengths.long() - 1)
        return self.normed(x[last].contiguous(), h[last].contiguous(), -1, fp8) @ self.head, states

    @torch.no_grad()
    def step(self, tokens, previous, states, slots, fp8=False):
        """Logits after one more token for each sequence (and the one before it); states[i][slots[b]] is sequence b's
        state of layer i."""
        x = self.inputs(tokens, previous)
        h = torch.zeros_like(x)
        for i in range(len(self.project)):
            o = mgs.mgs_linattn_step(*self.split(i, self.normed(x, h, i, fp8)), states[i], slots=slots,
                                     scale=self.key ** -0.5)
            x = o.flatten(1) @ self.back[i]
        return self.normed(x, h, -1, fp8) @ self.head


def phrases(batch, steps, phrase, vocab, gen):
    """Sequences that repeat a random phrase."""
    p = torch.randint(0, vocab, (batch, phrase), generator=gen)
    return p.repeat(1, -(-steps // phrase))[:, :steps].cuda()


def train(model, steps, batch=128, length=97, phrase=8, vocab=32, rate=5e-3, max_norm=1.0, seed=1, log=print):
    """Losses of `steps` steps of Adam on clipped gradients."""
    gen = torch.Generator().manual_seed(seed)
    params = list(model.parameters())
    optimizer = torch.optim.Adam(params, lr=rate)
    losses = []
    for n in range(steps):
        tokens = phrases(batch, length, phrase, vocab, gen)
        logits = model(tokens[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits.float().flatten(0, 1), tokens[:, 1:].flatten())
        optimizer.zero_grad()
        loss.backward()
        norm, _ = mgs.mgs_clip_norm([p.grad for p in params], max_norm)
        optimizer.step()
        losses.append(loss.item())
        if n % 20 == 0 or n == steps - 1:
            log(f"step {n:4d}  loss {losses[-1]:.4f}  gradient norm {norm.item():.3f}")
    return losses


def generate(model, tokens, lengths, count, fp8=False):
    """Greedy continuation of each prompt by `count` tokens, through a cache with more slots than sequences."""
    B = tokens.shape[0]
    logits, states = model.prompt(tokens, lengths, fp8)
    slots = torch.arange(B, 0, -1, dtype=torch.int32, device="cuda")   # in no particular order
    cache = []
    for S in states:
        c = S.new_zeros(B + 1, *S.shape[1:])
        c[slots.long()] = S
        cache.append(c)
    out = [tokens[torch.arange(B, device="cuda"), lengths.long() - 1], logits.argmax(-1)]
    while len(out) <= count:
        out.append(model.step(out[-1], out[-2], cache, slots, fp8).argmax(-1))
    return torch.stack(out[1:], 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--fp8", action="store_true")
    a = ap.parse_args(argv)
    model = Model()
    losses = train(model, a.steps)
    tokens = phrases(4, 60, 8, 32, torch.Generator().manual_seed(7))
    lengths = torch.tensor([40, 25, 48, 36], dtype=torch.int32, device="cuda")
    text = generate(model, tokens, lengths, 12, a.fp8)
    want = torch.stack([tokens[b, int(n):int(n) + 12] for b, n in enumerate(lengths)])
    right = float((text == want).float().mean())
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; {100 * right:.0f}% of the continuation right")
    return losses, right


if __name__ == "__main__":
    main()
