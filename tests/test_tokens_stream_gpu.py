"""The token path's operators on other streams than the current one, captured into graphs that are replayed, and run
together as a program runs them; what their binding refuses."""
import pytest
import torch

from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu


def inputs(dev, B=3, T=700, D=320, V=1000, dt=torch.bfloat16, seed=0):
    g = torch.Generator(dev).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    return dict(ids=torch.randint(-1, V, (B, T), generator=g, device=dev), W=rand(V, D).to(dt),
                x=rand(B, T, D).to(dt), r=rand(B, T, D).to(dt), i=rand(B, T, D).to(dt), dy=rand(B, T, D).to(dt),
                lam=rand(D) - 4, h=rand(B, D), logits=3 * rand(B, V), u=torch.rand(B, generator=g, device=dev),
                states=rand(B, -(-T // 64), D), logits16=3 * rand(B, V).bfloat16())


def calls(mgs, a):
    V = a["W"].shape[0]
    gates = (a["x"], a["r"], a["i"], a["lam"])
    return {
        "lookup": lambda **k: (mgs.mgs_embed_fwd(a["ids"], a["W"], **k),),
        "table": lambda **k: (mgs.mgs_embed_bwd(a["ids"], a["dy"], V, **k),),
        "gated": lambda **k: mgs.mgs_gated_fwd(*gates, want_states=True, **k),
        "gated_bwd": lambda **k: mgs.mgs_gated_bwd(*gates, a["dy"], a["states"], **k),
        "step": lambda **k: (mgs.mgs_gated_step(*(t[:, 0] for t in gates[:3]), a["lam"], a["h"], **k),),
        "sample": lambda **k: mgs.mgs_sample(a["logits"], a["u"], top_k=50, top_p=0.9, **k),
        "sample_bf16": lambda **k: mgs.mgs_sample(a["logits16"], a["u"], top_p=0.9, min_p=0.01, **k),
    }


NAMES = ["lookup", "table", "gated", "gated_bwd", "step", "sample", "sample_bf16"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream(gpu, name):
    import scan_linear_rnns_amd as mgs
    say(f"tokens {name} on a side stream")
    a = inputs(gpu)
    call = calls(mgs, a)[name]
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    keep = a["h"].clone()
    want = [t.clone() for t in call()]
    a["h"].copy_(keep)
    side.wait_stream(here)
    torch.cuda.synchronize()
    got = call(stream=side)
    torch.cuda.synchronize()
    owner = {b["address"]: seg["stream"] for seg in torch.cuda.memory_snapshot() for b in seg["blocks"]}
    assert {owner[t.data_ptr()] for t in got} == {side.cuda_stream}
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(gpu, name):
    """Captured once, replayed with other inputs in the same buffers and eager calls between: each replay is the eager
    result."""
    import scan_linear_rnns_amd as mgs
    say(f"tokens {name} in a graph")
    a = inputs(gpu)
    call = calls(mgs, a)[name]
    ws = {}
    if name.startswith("gated"):
        ws["ws"] = mgs.workspace(mgs.mgs_gated_workspace_size(3, 700, 320, dtype=torch.bfloat16, backward=True), gpu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(**ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(**ws)
    for n in range(4):
        for k, v in inputs(gpu, seed=n + 1).items():
            a[k].copy_(v)
        state = a["h"].clone()
        want = [t.clone() for t in call(**ws)]
        a["h"].copy_(state)
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(-7)
        graph.replay()
        a["junk"] = torch.randn(1 << 20, device=gpu).sum()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y), n


def test_two_graphs_on_one_workspace(gpu):
    """Calls of two sizes, captured into a graph each, all on one workspace, replayed in turn with eager calls between."""
    import scan_linear_rnns_amd as mgs
    say("tokens two graphs")
    both = [inputs(gpu, seed=1), inputs(gpu, B=1, T=5000, D=70, V=40000, dt=torch.float32, seed=2)]
    sizes = [mgs.mgs_gated_workspace_size(3, 700, 320, backward=True),
             mgs.mgs_gated_workspace_size(1, 5000, 70, backward=True),
             mgs.mgs_embed_workspace_size(2100, 1000, 320), mgs.mgs_embed_workspace_size(5000, 40000, 70),
             mgs.mgs_sample_workspace_size(3, 1000), mgs.mgs_sample_workspace_size(1, 40000)]
    # (the recurrence's words are tagged: its workspace is its own)
    spaces = {"gated": mgs.workspace(max(sizes[:2]), gpu), "other": mgs.workspace(max(sizes[2:]), gpu)}
    use = {"table": "other", "gated": "gated", "gated_bwd": "gated", "sample": "other"}

    def run(a):
        return [t for name, ws in use.items() for t in calls(mgs, a)[name](ws=spaces[ws])]

    want = [[t.clone() for t in run(a)] for a in both]
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in both], []
    for graph, a in zip(graphs, both):
        with torch.cuda.graph(graph):
            outs.append(run(a))
    for n in range(4):
        for k in ((0, 1), (1, 0), (0, 0), (1, 1))[n]:
            for o in outs[k]:
                o.fill_(-7)
            graphs[k].replay()
            got = run(both[1 - k])   # eager, on the same workspaces
            torch.cuda.synchronize()
            for x, y in zip(outs[k], want[k]):
                assert torch.equal(x, y), (n, k)
            for x, y in zip(got, want[1 - k]):
                assert torch.equal(x, y), (n, k)
    assert mgs.mgs_workspace_check(spaces["gated"]) == 0


def test_two_streams_at_once(gpu):
    """The same operators on two streams, a workspace each, interleaved."""
    import scan_linear_rnns_amd as mgs
    say("tokens two streams")
    both = [inputs(gpu, seed=s) for s in (1, 2)]
    todo = [calls(mgs, a) for a in both]
    want = [[t.clone() for name in NAMES if name != "step" for t in c[name]()] for c in todo]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        got = [[], []]
        for name in NAMES:
            if name != "step":
                for k in (0, 1):
                    got[k] += todo[k][name](stream=streams[k])
    torch.cuda.synchronize()
    for k in (0, 1):
        for x, y in zip(got[k], want[k]):
            assert torch.equal(x, y)


class Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, W):
        import scan_linear_rnns_amd as mgs
        ctx.save_for_backward(ids)
        ctx.vocab = W.shape[0]
        return mgs.mgs_embed_fwd(ids, W, scale=2.0)

    @staticmethod
    def backward(ctx, dy):
        import scan_linear_rnns_amd as mgs
        return None, mgs.mgs_embed_bwd(*ctx.saved_tensors, dy.contiguous(), ctx.vocab, scale=2.0)


class Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, lam, reset):
        import scan_linear_rnns_amd as mgs
        y, _, states = mgs.mgs_gated_fwd(x, r, i, lam, reset=reset, want_state=False, want_states=True)
        ctx.save_for_backward(x, r, i, lam, reset, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        import scan_linear_rnns_amd as mgs
        x, r, i, lam, reset, states = ctx.saved_tensors
        return (*mgs.mgs_gated_bwd(x, r, i, lam, dy.contiguous(), states, reset=reset, want_dh0=False)[:4], None)


def test_a_run_of_them(gpu):
    """Lookup, a projection, the recurrence on packed documents and the logits, their gradients against the same in
    torch in 64 bits; then the last tokens' distribution is drawn from, and the next step goes on from there."""
    import scan_linear_rnns_amd as mgs
    say("tokens together")
    B, T, D, V = 2, 150, 48, 90
    g = torch.Generator(gpu).manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device=gpu)  # noqa: E731
    ids = torch.randint(0, V, (B, T), generator=g, device=gpu)
    reset = torch.rand(B, T, generator=g, device=gpu) < 0.02
    leaves = [rand(V, D), rand(D, 3 * D) * D ** -0.5, rand(D) - 4, rand(D, V) * D ** -0.5]
    dlogits = rand(B, T, V)

    def forward(W, P, lam, head, lookup, gated):
        x, r, i = (lookup(ids, W) @ P).split(D, dim=2)
        return gated(x, r, i, lam, reset) @ head

    def gated64(x, r, i, lam, reset):
        log_a = -8.0 * torch.nn.functional.softplus(lam) * torch.sigmoid(r)
        new = reset[:, :, None]
        a = torch.exp(log_a).masked_fill(new, 0.0)
        b = torch.sqrt(-torch.expm1(2 * log_a)).masked_fill(new, 1.0) * torch.sigmoid(i) * x
        h, rows = torch.zeros_like(x[:, 0]), []
        for t in range(T):
            h = a[:, t] * h + b[:, t]
            rows.append(h)
        return torch.stack(rows, 1)

    own = [t.clone().requires_grad_() for t in leaves]
    logits = forward(*own, Lookup.apply, Gated.apply)
    grads = torch.autograd.grad(logits, own, dlogits)
    exact = [t.double().requires_grad_() for t in leaves]
    want = forward(*exact, lambda n, W: 2.0 * W[n], gated64)
    wants = torch.autograd.grad(want, exact, dlogits.double())
    # products of 48 and 144 terms and a recurrence, in 32 bits: some hundreds of 2^-24 of the largest
    for x, y in zip((logits, *grads), (want, *wants)):
        assert (x.double() - y).abs().max() <= 500 * 2.0 ** -24 * y.abs().max()

    u = torch.rand(B, generator=g, device=gpu)
    token, logp = mgs.mgs_sample(logits[:, -1].detach(), u, temperature=0.7)
    p = torch.softmax(logits[:, -1].double() / 0.7000000000000001, 1)
    assert (torch.log(p.gather(1, token[:, None])[:, 0]) - logp).abs().max() < 1e-5
    W, P, lam, _ = leaves
    x, r, i = (mgs.mgs_embed_fwd(ids, W, scale=2.0) @ P).split(D, dim=2)
    _, state, _ = mgs.mgs_gated_fwd(x, r, i, lam, reset=reset)
    more = torch.cat([ids, token[:, None]], 1)
    x, r, i = (mgs.mgs_embed_fwd(more, W, scale=2.0) @ P).split(D, dim=2)
    whole, _, _ = mgs.mgs_gated_fwd(x, r, i, lam, reset=torch.nn.functional.pad(reset, (0, 1)))
    y = mgs.mgs_gated_step(x[:, -1], r[:, -1], i[:, -1], lam, state)
    assert (y - whole[:, -1]).abs().max() <= 1e-5 * whole.abs().max()


def test_refusals_of_the_binding(gpu):
    import scan_linear_rnns_amd as mgs
    say("tokens refusals")
    a = inputs(gpu, T=70)
    gates = (a["x"], a["r"], a["i"], a["lam"])
    cpu = a["x"].cpu()
    for bad, kind in (
            (lambda: mgs.mgs_embed_fwd(a["ids"].float(), a["W"]), TypeError),
            (lambda: mgs.mgs_embed_fwd(a["ids"].cpu(), a["W"]), TypeError),
            (lambda: mgs.mgs_embed_fwd(a["ids"], a["W"].half()), TypeError),
            (lambda: mgs.mgs_embed_fwd(a["ids"], a["W"].t()), ValueError),
            (lambda: mgs.mgs_embed_fwd(a["ids"].t(), a["W"]), ValueError),
            (lambda: mgs.mgs_embed_bwd(a["ids"][:, 1:].contiguous(), a["dy"], 10), ValueError),
            (lambda: mgs.mgs_embed_bwd(a["ids"], a["dy"], 10, accumulate=True), ValueError),
            (lambda: mgs.mgs_embed_bwd(a["ids"], a["dy"], 10, dW=a["W"]), ValueError),
            (lambda: mgs.mgs_gated_fwd(cpu, *gates[1:]), TypeError),
            (lambda: mgs.mgs_gated_fwd(a["x"], a["r"].float(), *gates[2:]), TypeError),
            (lambda: mgs.mgs_gated_fwd(a["x"], a["r"][:, 1:], *gates[2:]), ValueError),
            (lambda: mgs.mgs_gated_fwd(*gates[:3], a["lam"].bfloat16()), TypeError),
            (lambda: mgs.mgs_gated_fwd(*gates, reset=a["ids"]), TypeError),
            (lambda: mgs.mgs_gated_fwd(*gates, lengths=a["u"]), TypeError),
            (lambda: mgs.mgs_gated_fwd(*gates, rate=-1.0), mgs.MgsError),
            (lambda: mgs.mgs_gated_bwd(*gates, a["dy"], a["states"][:, 1:].contiguous()), ValueError),
            (lambda: mgs.mgs_gated_fwd(*gates, h0=a["h"], hT=a["h"]), mgs.MgsError),
            (lambda: mgs.mgs_gated_step(*gates, a["h"]), ValueError),
            (lambda: mgs.mgs_gated_step(*(t[:, 0] for t in gates[:3]), a["lam"], a["h"][:2]), mgs.MgsError),
            (lambda: mgs.mgs_sample(a["logits"][0], a["u"]), ValueError),
            (lambda: mgs.mgs_sample(a["logits"], a["u"].double()), TypeError),
            (lambda: mgs.mgs_sample(a["logits"], a["u"], top_k=torch.zeros(3, device=gpu)), TypeError),
            (lambda: mgs.mgs_sample(a["logits"], a["u"], top_p=torch.zeros(2, device=gpu)), ValueError),
            (lambda: mgs.mgs_sample(a["logits"], a["u"], temperature=torch.ones(3)), TypeError),
            (lambda: mgs.mgs_sample(a["logits"], a["u"], ws=torch.zeros(8, dtype=torch.uint8, device=gpu)), mgs.MgsError),
            (lambda: mgs.mgs_gated_fwd(*gates, ws=torch.zeros(8, dtype=torch.uint8, device=gpu)), mgs.MgsError)):
        with pytest.raises(kind):
            bad()
    torch.cuda.synchronize()
