"""A small recurrent language model on the token path's operators: trained on packed documents, then sampled from.

    python examples/gated_lm.py [--steps 200] [--temperature 0.8] [--top-k 20] [--top-p 0.95]

Tokens are looked up in a scaled table (mgs_embed_fwd, _bwd); each layer adds what came before to the residual stream and
norms the sum (mgs_rmsnorm_fwd, _bwd), projects it to the inputs and gates of the gated linear recurrence
(mgs_gated_fwd, _bwd), which starts anew at each document, and projects back.  Training clips the gradients by their
global norm (mgs_clip_norm).  Generation reads prompts of unlike lengths in one pass, keeps each sequence's states in a
cache, and draws one token at a time (mgs_gated_step, mgs_sample).

The data are synthetic: documents that repeat a random phrase, several to a sequence.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import scan_linear_rnns_amd as mgs  # noqa: E402
from recurrent_lm import EPS, AddNorm  # noqa: E402

RATE = 8.0


class Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.table, ctx.scale = table, scale
        return mgs.mgs_embed_fwd(ids, table, scale=scale)

    @staticmethod
    def backward(ctx, dy):
        table = ctx.table
        return None, mgs.mgs_embed_bwd(*ctx.saved_tensors, dy.contiguous(), table.shape[0], scale=ctx.scale,
                                       dtype=table.dtype), None


class Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, lam, reset):
        y, _, states = mgs.mgs_gated_fwd(x, r, i, lam, reset=reset, rate=RATE, want_state=False, want_states=True)
        ctx.save_for_backward(x, r, i, lam, reset, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, r, i, lam, reset, states = ctx.saved_tensors
        grads = mgs.mgs_gated_bwd(x, r, i, lam, dy.contiguous(), states, reset=reset, rate=RATE, want_dh0=False)
        return (*grads[:4], None)


class Model(torch.nn.Module):
    def __init__(self, vocab=32, width=128, layers=2, dtype=torch.float32, seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape, std):
            return torch.nn.Parameter((std * torch.randn(*shape, generator=gen)).to(device="cuda", dtype=dtype))

        self.width = width
        self.table = weight(vocab, width, std=width ** -0.5)
        self.project = torch.nn.ParameterList([weight(width, 4 * width, std=width ** -0.5) for _ in range(layers)])
        self.back = torch.nn.ParameterList([weight(width, width, std=width ** -0.5) for _ in range(layers)])
        self.norms = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(width, device="cuda", dtype=dtype))
                                             for _ in range(layers + 1)])
        # decays between 0.5 and 0.999 with the gate open; the parameter is float32 whatever the others are
        most = 0.5 + 0.499 * torch.rand(layers, width, generator=gen)
        self.lam = torch.nn.ParameterList([torch.nn.Parameter(z.cuda())
                                           for z in torch.log(torch.expm1(-torch.log(most) / RATE))])
        self.head = weight(width, vocab, std=width ** -0.5)

    def split(self, i, y):
        """Layer i's inputs, gates (views of one projection) and output gate of normed inputs y (...,width)."""
        x, r, g, z = torch.split(y @ self.project[i], self.width, dim=-1)
        return x, r, g, torch.nn.functional.silu(z)

    def forward(self, tokens, reset):
        x = Lookup.apply(tokens, self.table, math.sqrt(self.width))
        h = torch.zeros_like(x)
        for i in range(len(self.project)):
            y, h = AddNorm.apply(x, h, self.norms[i])
            x, r, g, z = self.split(i, y)
            x = (Gated.apply(x, r, g, self.lam[i], reset) * z) @ self.back[i]
        y, _ = AddNorm.apply(x, h, self.norms[-1])
        return y @ self.head

    # ---- generation

    def normed(self, x, h, i):
        """The norm without a gradient; the residual stream h is updated in place."""
        return mgs.mgs_rmsnorm_fwd(x, self.norms[i], h, eps=EPS, h=h)[0]

    @torch.no_grad()
    def prompt(self, tokens, lengths):
        """Reads prompts of unlike lengths; logits after each one's last token, and the states."""
        x = mgs.mgs_embed_fwd(tokens, self.table, scale=math.sqrt(self.width))
        h, states = torch.zeros_like(x), []
        for i in range(len(self.project)):
            x, r, g, z = self.split(i, self.normed(x, h, i))
            y, hT, _ = mgs.mgs_gated_fwd(x, r, g, self.lam[i], lengths=lengths, rate=RATE)
            states.append(hT)
            x = (y * z) @ self.back[i]
        last = (torch.arange(tokens.shape[0], device="cuda"), lengths.long() - 1)
        return self.normed(x[last].contiguous(), h[last].contiguous(), -1) @ self.head, states

    @torch.no_grad()
    def step(self, tokens, states, slots):
        """Logits after one more token for each sequence; states[i][slots[b]] is sequence b's state of layer i."""
        x = mgs.mgs_embed_fwd(tokens, self.table, scale=math.sqrt(self.width))
        h = torch.zeros_like(x)
        for i in range(len(self.project)):
            x, r, g, z = self.split(i, self.normed(x, h, i))
            x = (mgs.mgs_gated_step(x, r, g, self.lam[i], states[i], slots=slots, rate=RATE) * z) @ self.back[i]
        return self.normed(x, h, -1) @ self.head


def documents(batch, steps, vocab, gen, phrase=4, length=40):
    """Sequences of documents that each repeat a random phrase, and where the documents start."""
    count = -(-steps // length)
    p = torch.randint(0, vocab, (batch, count, phrase), generator=gen).repeat(1, 1, -(-length // phrase))[:, :, :length]
    starts = torch.zeros(batch, count, length, dtype=torch.bool)
    starts[:, :, 0] = True
    return p.flatten(1)[:, :steps].cuda(), starts.flatten(1)[:, :steps].cuda()


def loss_of(model, tokens, reset):
    """Mean cross entropy of each token after the one before, but for those that start a document."""
    logits = model(tokens[:, :-1].contiguous(), reset[:, :-1].contiguous())
    target = tokens[:, 1:].masked_fill(reset[:, 1:], -100)
    return torch.nn.functional.cross_entropy(logits.float().flatten(0, 1), target.flatten())


def train(model, steps, batch=64, length=161, vocab=32, rate=3e-3, max_norm=1.0, seed=1, log=print):
    """Losses of `steps` steps of Adam on clipped gradients."""
    gen = torch.Generator().manual_seed(seed)
    params = list(model.parameters())
    optimizer = torch.optim.Adam(params, lr=rate)
    losses = []
    for n in range(steps):
        loss = loss_of(model, *documents(batch, length, vocab, gen))
        optimizer.zero_grad()
        loss.backward()
        norm, _ = mgs.mgs_clip_norm([p.grad for p in params], max_norm)
        optimizer.step()
        losses.append(loss.item())
        if n % 20 == 0 or n == steps - 1:
            log(f"step {n:4d}  loss {losses[-1]:.4f}  gradient norm {norm.item():.3f}")
    return losses


def generate(model, tokens, lengths, count, gen, **settings):
    """Continues each prompt by `count` drawn tokens, through a cache with more slots than sequences; the tokens and
    the logs of their shares of the kept weight."""
    B = tokens.shape[0]
    logits, states = model.prompt(tokens, lengths)
    slots = torch.arange(B, 0, -1, dtype=torch.int32, device="cuda")   # in no particular order
    cache = []
    for S in states:
        c = S.new_zeros(B + 1, S.shape[1])
        c[slots.long()] = S
        cache.append(c)
    out, logs = [], []
    for _ in range(count):
        u = torch.rand(B, generator=gen, device="cuda")
        token, logp = mgs.mgs_sample(logits, u, **settings)
        out.append(token)
        logs.append(logp)
        logits = model.step(token, cache, slots)
    return torch.stack(out, 1), torch.stack(logs, 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-k", type=int, default=20)
    ap.add_argument("--top-p", type=float, default=0.95)
    a = ap.parse_args(argv)
    model = Model()
    losses = train(model, a.steps)
    tokens, _ = documents(4, 40, 32, torch.Generator().manual_seed(7))
    lengths = torch.tensor([40, 25, 38, 36], dtype=torch.int32, device="cuda")
    text, logs = generate(model, tokens, lengths, 12, torch.Generator("cuda").manual_seed(3), temperature=a.temperature,
                          top_k=a.top_k, top_p=a.top_p)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    for row, log in zip(text.tolist(), logs.sum(1).tolist()):
        print(" ".join(f"{t:2d}" for t in row), f"  log probability {log:.2f}")
    return losses, text


if __name__ == "__main__":
    main()
