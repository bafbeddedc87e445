"""GPU parity of linear attention with a decay per head (mgs_linattn_fwd, _bwd, _step) with the step-by-step
recurrence in 64 bits.

Tolerance, element by element: every output is a sum of products, and a sum of n terms in fp32 is off by at most
n 2^-24 times the sum of the terms' absolute values (which the reference gives on absolute inputs).  The terms pass a
dot product over dk or dv, a chunk of 64 steps, one addition a chunk, and a decay, whose exponent is good to 2^-24 of
itself (under 40 where the decay counts): n = dk + dv + 64 + chunks + 48.  An output in bf16 is rounded once more, by
at most 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from tests import layers_reference as ref
from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(dev, B, T, H, Hk, dk, dv, dtype="f32", decay="step", S0=False, lengths=None, fused=False, seed=0, back=True):
    """Inputs on the GPU, and the same values in 64 bits for the reference."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    parts = [rand(B, T, Hk * dk), rand(B, T, Hk * dk) * dk ** -0.5, rand(B, T, H * dv)]
    if fused:
        both = torch.cat(parts, 2).to(DT[dtype]).to(dev)
        q, k, v = torch.split(both, [Hk * dk, Hk * dk, H * dv], dim=2)
    else:
        q, k, v = (p.to(DT[dtype]).to(dev) for p in parts)
    a = dict(q=q.unflatten(2, (Hk, dk)), k=k.unflatten(2, (Hk, dk)), v=v.unflatten(2, (H, dv)))
    rate = torch.logspace(-3, 0.3, H)
    a["g"] = (-rate if decay == "head" else -rate * rand(B, T, H).abs()).to(dev)
    a["S0"] = rand(B, H, dv, dk).to(dev) if S0 else None
    a["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev) if lengths is not None else None
    if back:
        a["do"] = rand(B, T, H, dv).to(DT[dtype]).to(dev)
        a["dST"] = rand(B, H, dv, dk).to(dev) if S0 else None
    return a


def reference(a, scale):
    b = {n: n64(t) if n != "lengths" else (None if t is None else t.cpu().numpy()) for n, t in a.items()}
    return ref.linattn(**b, scale=scale), ref.linattn_abs(**b, scale=scale)


def check(got, a, scale, who=""):
    want, size = reference(a, scale)
    T, dk, dv = a["q"].shape[1], a["q"].shape[3], a["v"].shape[3]
    gamma = (dk + dv + 64 + -(-T // 64) + 48) * 2.0 ** -24
    for name, t in got.items():
        x = n64(t)
        tol = gamma * size[name] + (2.0 ** -8 * np.abs(want[name]) if t.dtype == torch.bfloat16 else 0.0)
        assert x.shape == want[name].shape, (who, name, x.shape, want[name].shape)
        far, norm = np.linalg.norm(x - want[name]), np.linalg.norm(want[name])
        if not (name == "dg" and a["g"].dim() == 1):   # a sum over steps whose terms may cancel
            assert far <= (2.0 ** -8 if t.dtype == torch.bfloat16 else 2e-5) * norm, (who, name, far, norm)
        bad = ~(np.abs(x - want[name]) <= tol)
        assert not bad.any(), (who, name, int(bad.sum()), float(np.abs(x - want[name])[bad].max()), float(np.min(np.broadcast_to(tol, x.shape)[bad])))


def run(a, scale, **more):
    import scan_linear_rnns_amd as mgs
    ins = [a[n] for n in ("q", "k", "v", "g")]
    o, ST, _ = mgs.mgs_linattn_fwd(*ins, S0=a["S0"], lengths=a["lengths"], scale=scale, **more)
    got = dict(o=o, ST=ST)
    if "do" in a:
        grads = mgs.mgs_linattn_bwd(*ins, a["do"], S0=a["S0"], dST=a["dST"], lengths=a["lengths"], scale=scale, **more)
        got.update(zip(("dq", "dk", "dv", "dg", "dS0"), grads))
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 129, 300])
def test_lengths(gpu, T, dtype):
    say(f"linattn T={T} {dtype}")
    a = make(gpu, 2, T, 2, 2, 64, 64, dtype, S0=True, seed=T)
    check(run(a, 0.125), a, 0.125)


DIMS = [(64, 64), (128, 128), (64, 128), (128, 64), (32, 48), (40, 104), (16, 8), (8, 128), (72, 64),
        (33, 17), (1, 1), (127, 5), (2, 65)]   # the last four have no aligned rows


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_head_dims(gpu, dk, dv, dtype):
    say(f"linattn dk={dk} dv={dv} {dtype}")
    a = make(gpu, 1, 130, 2, 1, dk, dv, dtype, S0=True, seed=dk + dv)
    check(run(a, dk ** -0.5), a, dk ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["step", "head"])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (4, 1), (6, 2)])
def test_heads_and_decays(gpu, H, Hk, decay, dtype):
    say(f"linattn H={H} Hk={Hk} decay per {decay} {dtype}")
    a = make(gpu, 2, 150, H, Hk, 64, 64, dtype, decay=decay, seed=H)
    check(run(a, 0.125), a, 0.125)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,d", [(1, 2100, 64), (3, 1030, 128), (1, 4500, 32)])
def test_long_sequences_are_cut(gpu, B, T, d, dtype):
    """Few heads and many steps: segments, chained, in both directions; the last one ragged."""
    say(f"linattn long B={B} T={T} d={d} {dtype}")
    a = make(gpu, B, T, 1, 1, d, d, dtype, S0=True, seed=T)
    check(run(a, d ** -0.5), a, d ** -0.5)


def test_many_heads_are_not_cut(gpu):
    """Enough (sequence, head) pairs to fill the chip: the forward walks each sequence in one piece."""
    import scan_linear_rnns_amd as mgs
    say("linattn B=64 T=140 H=8")
    assert mgs.mgs_linattn_workspace_size(64, 140, 8, 8, 32, 32) <= 256
    a = make(gpu, 64, 140, 8, 8, 32, 32, "f32", S0=True, seed=5)
    check(run(a, 0.2), a, 0.2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ragged_batch_does_not_read_padding(gpu, dtype):
    """Lengths of zero, one, a chunk's edge, past T; NaN and infinities in every padded place."""
    T, lengths = 200, [0, 1, 64, 65, 200, 131, 1000, -3]
    say(f"linattn ragged {dtype}")
    a = make(gpu, 8, T, 2, 1, 64, 64, dtype, S0=True, lengths=lengths, seed=3)
    clean = {n: t for n, t in a.items()}
    dirty = dict(a)
    for n in ("q", "k", "v", "g", "do"):
        dirty[n] = a[n].clone()
        for b, m in enumerate(lengths):
            m = max(0, m)
            dirty[n][b, m:] = float("nan")
            dirty[n][b, m + 1::3] = float("-inf")
    got = run(dirty, 0.125)
    check(got, clean, 0.125)
    for n in ("o", "dq", "dk", "dv", "dg"):
        for b, m in enumerate(lengths):
            assert torch.count_nonzero(got[n][b, max(0, m):]) == 0, (n, b)
    assert torch.equal(got["ST"][0], a["S0"][0]) and torch.equal(got["dS0"][0], a["dST"][0])


def test_strided_inputs(gpu):
    """Views of one projection, heads ahead of steps, broadcast inputs, rows that no wide access may take."""
    import scan_linear_rnns_amd as mgs
    say("linattn strides")
    for dtype in ("f32", "bf16"):
        a = make(gpu, 2, 100, 4, 2, 64, 64, dtype, fused=True, seed=9)
        check(run(a, 0.125), a, 0.125, "fused")
        b = dict(a)
        for n in ("q", "k", "v", "do"):
            b[n] = a[n].transpose(1, 2).contiguous().transpose(1, 2)
        b["g"] = a["g"].transpose(1, 2).contiguous().transpose(1, 2)
        check(run(b, 0.125), a, 0.125, "heads first")
        c = dict(a)
        for n in ("q", "k", "v", "do"):
            pad = torch.empty(*a[n].shape[:3], a[n].shape[3] + 3, dtype=a[n].dtype, device=gpu)
            pad[..., 1:-2] = a[n]
            c[n] = pad[..., 1:-2]
        check(run(c, 0.125), a, 0.125, "unaligned")
        e = dict(a, v=a["v"][:, :1].expand(-1, 100, -1, -1), g=a["g"][:1].expand(2, -1, -1))
        check(run(e, 0.125), {n: (t.contiguous() if n in ("v", "g") else t) for n, t in e.items()}, 0.125, "broadcast")
    assert mgs.mgs_linattn_workspace_size(2, 100, 4, 2, 64, 64, torch.float32) > 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_decays(gpu, dtype):
    """Cleared states (-inf), decays too small for fp32, none at all; a cleared step's dg is an exact zero."""
    say(f"linattn extreme decays {dtype}")
    a = make(gpu, 2, 700, 2, 2, 64, 64, dtype, S0=True, seed=11)
    g = a["g"]
    g[0, ::37] = float("-inf")
    g[0, 5:8] = float("-inf")
    g[1, :, 0] = 0.0
    g[1, 3::50, 1] = -3.0e38
    g[1, 7::50, 1] = -150.0
    got = run(a, 0.125)
    check(got, a, 0.125)
    assert torch.count_nonzero(got["dg"][g < -104]) == 0
    a["g"] = torch.full_like(g, float("-inf"))      # every step forgets everything before it
    got = run(a, 0.125)
    check(got, a, 0.125)
    assert torch.count_nonzero(got["dS0"]) == 0 and torch.count_nonzero(got["dg"]) == 0


def test_non_finite_inputs_propagate(gpu):
    say("linattn non-finite")
    for dtype in ("f32", "bf16"):
        a = make(gpu, 1, 200, 1, 1, 64, 64, dtype, back=False, seed=13)
        a["v"][0, 70, 0, 3] = float("nan")
        o = run(a, 1.0)["o"].float()
        assert torch.isfinite(o[0, :70]).all() and not torch.isfinite(o[0, 70:, 0, 3]).any()
        assert torch.isfinite(o[..., 4:]).all()
        a["v"][0, 70, 0, 3] = 0.0
        a["g"][0, 100] = float("nan")
        o = run(a, 1.0)["o"].float()
        assert torch.isfinite(o[0, :100]).all() and torch.isnan(o[0, 100:]).all()


def test_empty(gpu):
    import scan_linear_rnns_amd as mgs
    say("linattn T = 0, B = 0")
    a = make(gpu, 2, 0, 2, 1, 32, 32, S0=True)
    got = run(a, 1.0)
    assert torch.equal(got["ST"], a["S0"]) and torch.equal(got["dS0"], a["dST"]) and got["o"].numel() == 0
    a = make(gpu, 2, 0, 2, 1, 32, 32, decay="head")
    got = run(a, 1.0)
    assert torch.count_nonzero(got["ST"]) == 0 and torch.count_nonzero(got["dg"]) == 0
    assert run(make(gpu, 0, 5, 2, 1, 32, 32), 1.0)["o"].shape == (0, 5, 2, 32)
    o = mgs.mgs_linattn_step(torch.empty(0, 1, 32, device=gpu), torch.empty(0, 1, 32, device=gpu),
                             torch.empty(0, 2, 32, device=gpu), torch.empty(0, 2, device=gpu),
                             torch.zeros(3, 2, 32, 32, device=gpu))
    assert o.shape == (0, 2, 32)


def test_runs_alike_every_time(gpu):
    say("linattn determinism")
    a = make(gpu, 2, 1500, 4, 2, 128, 128, "bf16", S0=True, seed=17)
    first = {n: t.clone() for n, t in run(a, 0.1).items()}
    for _ in range(3):
        for n, t in run(a, 0.1).items():
            assert torch.equal(first[n], t), n


def test_gradient_against_differences(gpu):
    """L is linear in q, k, v and S0 one at a time, so a central difference has no truncation at any step; what is left
    is the rounding of two fp32 forwards, gamma times the sum of absolute terms."""
    import scan_linear_rnns_amd as mgs
    say("linattn differences")
    a = make(gpu, 2, 200, 2, 2, 64, 64, "f32", S0=True, seed=19)
    got = run(a, 0.125)

    def loss(**change):
        b = {**a, **change}
        o, ST, _ = mgs.mgs_linattn_fwd(b["q"], b["k"], b["v"], b["g"], S0=b["S0"], scale=0.125)
        return float((o.double() * a["do"].double()).sum() + (ST.double() * a["dST"].double()).sum())

    for i, n in enumerate(("q", "k", "v", "S0")):
        u = torch.randn(a[n].shape, generator=torch.Generator().manual_seed(i)).to(gpu)
        diff = (loss(**{n: a[n] + u}) - loss(**{n: a[n] - u})) / 2
        up = {**a, n: (a[n].abs() + u.abs())}
        _, size = reference(up, 0.125)
        total = (size["o"] * np.abs(n64(a["do"]))).sum() + (size["ST"] * np.abs(n64(a["dST"]))).sum()
        tol = 2 * (64 + 64 + 64 + 4 + 48) * 2.0 ** -24 * total
        assert abs(diff - float((got["d" + n].double() * u.double()).sum())) <= tol, (n, diff, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (5, 2, 2, 40, 72), (2, 3, 1, 33, 17),
                                          (7, 2, 1, 128, 8), (40, 8, 8, 64, 128)])
def test_step(gpu, B, H, Hk, dk, dv, dtype):
    import scan_linear_rnns_amd as mgs
    say(f"linattn step B={B} H={H} Hk={Hk} dk={dk} dv={dv} {dtype}")
    a = make(gpu, B, 1, H, Hk, dk, dv, dtype, S0=True, seed=B, back=False)
    want, size = reference(a, 0.3)
    n_slots = B + 3
    slots = torch.randperm(n_slots, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32).to(gpu)
    S = torch.full((n_slots, H, dv, dk), 7.0, device=gpu)
    S[slots.long()] = a["S0"]
    if B > 2:
        slots[1] = -1
    before = S.clone()
    o = mgs.mgs_linattn_step(a["q"][:, 0], a["k"][:, 0], a["v"][:, 0], a["g"][:, 0], S, slots=slots, scale=0.3)
    gamma = (dk + 48) * 2.0 ** -24
    for b in range(B):
        if slots[b] < 0:
            assert torch.count_nonzero(o[b]) == 0
            continue
        for x, name in ((o[b], "o"), (S[slots[b].long()], "ST")):
            w, s = (want["o"][b, 0], size["o"][b, 0]) if name == "o" else (want["ST"][b], size["ST"][b])
            tol = gamma * s + (2.0 ** -8 * np.abs(w) if x.dtype == torch.bfloat16 else 0.0)
            assert (np.abs(n64(x) - w) <= tol).all(), (name, b)
    idle = torch.ones(n_slots, dtype=torch.bool, device=gpu)
    idle[slots[slots >= 0].long()] = False
    assert torch.equal(S[idle], before[idle])


def test_step_continues_a_prompt(gpu):
    """A prompt, then single steps from its state, against the whole sequence."""
    import scan_linear_rnns_amd as mgs
    say("linattn prompt then steps")
    a = make(gpu, 2, 90, 4, 2, 64, 64, "f32", back=False, seed=23)
    _, S, _ = mgs.mgs_linattn_fwd(*(a[n][:, :77] for n in ("q", "k", "v", "g")), scale=0.125)
    o = [mgs.mgs_linattn_step(a["q"][:, t], a["k"][:, t], a["v"][:, t], a["g"][:, t], S, scale=0.125)
         for t in range(77, 90)]
    want, size = reference(a, 0.125)
    gamma = (64 + 64 + 64 + 2 + 48 + 13) * 2.0 ** -24
    assert (np.abs(n64(torch.stack(o, 1)) - want["o"][:, 77:]) <= gamma * size["o"][:, 77:]).all()
    assert (np.abs(n64(S) - want["ST"]) <= gamma * size["ST"]).all()


def test_step_in_a_cache_past_32_bit_offsets(gpu):
    """A cache of over 2^31 elements: the last slot's state, at an offset past 32 bits, and the first."""
    import scan_linear_rnns_amd as mgs
    H, d = 8, 128
    n_slots = (1 << 31) // (H * d * d) + 3
    say(f"linattn step, cache of {n_slots * H * d * d} elements")
    a = make(gpu, 2, 1, H, H, d, d, "bf16", S0=True, seed=29, back=False)
    S = torch.empty(n_slots, H, d, d, device=gpu)
    slots = torch.tensor([n_slots - 1, 0], dtype=torch.int32, device=gpu)
    S[slots.long()] = a["S0"]
    S[1] = 5.0
    mgs.mgs_linattn_step(a["q"][:, 0], a["k"][:, 0], a["v"][:, 0], a["g"][:, 0], S, slots=slots)
    want, size = reference(a, 1.0)
    assert (np.abs(n64(S[slots.long()]) - want["ST"]) <= (d + 48) * 2.0 ** -24 * size["ST"]).all()
    assert bool((S[1] == 5.0).all())


def test_other_stream_and_graph_replays(gpu):
    """The calls run on the stream they are given, and a captured graph replays to the eager results."""
    import scan_linear_rnns_amd as mgs
    say("linattn streams and graphs")
    a = make(gpu, 1, 1100, 2, 1, 64, 64, "bf16", S0=True, seed=31)
    ref_out = {n: t.clone() for n, t in run(a, 0.125).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(a, 0.125, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for n in ref_out:
        assert torch.equal(ref_out[n], got[n]), n
    ins = [a[n] for n in ("q", "k", "v", "g")]
    dims = (1, 1100, 2, 1, 64, 64)
    ws = mgs.workspace(mgs.mgs_linattn_workspace_size(*dims, dtype=torch.bfloat16, backward=True), gpu)
    outs = {n: torch.empty_like(t) for n, t in ref_out.items()}
    S = a["S0"].clone()
    so = torch.empty(1, 2, 64, dtype=torch.bfloat16, device=gpu)
    step = [a[n][:, 0].contiguous() for n in ("q", "k", "v", "g")]

    def work():
        S.copy_(a["S0"])
        mgs.mgs_linattn_step(*step, S, o=so)
        mgs.mgs_linattn_fwd(*ins, S0=a["S0"], scale=0.125, o=outs["o"], ST=outs["ST"], ws=ws)
        mgs.mgs_linattn_bwd(*ins, a["do"], S0=a["S0"], dST=a["dST"], scale=0.125, ws=ws,
                            out=tuple(outs[n] for n in ("dq", "dk", "dv", "dg", "dS0")))

    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    eager_S, eager_o = S.clone(), so.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        for t in outs.values():
            t.fill_(float("nan"))
        (torch.randn(1 << 18, device=gpu) * 2).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ref_out:
            assert torch.equal(ref_out[n], outs[n]), n
        assert torch.equal(S, eager_S) and torch.equal(so, eager_o)


def test_binding_refuses(gpu):
    import scan_linear_rnns_amd as mgs
    say("linattn refusals")
    a = make(gpu, 1, 8, 2, 1, 32, 32, back=False)
    q, k, v, g = (a[n] for n in ("q", "k", "v", "g"))
    for bad, err in (((q.half(), k.half(), v.half(), g), TypeError), ((q.cpu(), k, v, g), TypeError),
                     ((q, k, v, g.bfloat16()), TypeError), ((q, k[:, :4], v, g), ValueError),
                     ((q.transpose(2, 3), k, v, g), ValueError), ((q, k, v, g[..., :1]), ValueError),
                     ((q.bfloat16(), k, v, g), TypeError), ((q, k, v, None), ValueError)):
        with pytest.raises(err):
            mgs.mgs_linattn_fwd(*bad)
    wide = torch.zeros(1, 8, 1, 129, device=gpu)
    with pytest.raises(mgs.MgsError, match="UNSUPPORTED"):
        mgs.mgs_linattn_fwd(wide, wide, v, g)
    three = torch.zeros(1, 8, 3, 32, device=gpu)
    with pytest.raises(mgs.MgsError, match="INVALID"):       # 2 heads over 3 query/key heads
        mgs.mgs_linattn_fwd(three, three, v, g)
    with pytest.raises(mgs.MgsError, match="WORKSPACE"):
        mgs.mgs_linattn_bwd(q, k, v, g, torch.zeros_like(v), ws=torch.empty(256, dtype=torch.uint8, device=gpu))
    with pytest.raises(mgs.MgsError, match="INVALID"):       # more sequences than states, and no slots
        mgs.mgs_linattn_step(*(t.expand(4, *t.shape[1:]).contiguous() for t in (q[:, 0], k[:, 0], v[:, 0], g[:, 0])),
                             torch.zeros(3, 2, 32, 32, device=gpu))
    torch.cuda.synchronize()
