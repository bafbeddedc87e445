"""GPU tests of linear attention (mgs_linattn_fwd, _bwd, _step) at edges of its definition: empty batches, cleared
states, variants that only some calls reach.  Tolerances as in test_linattn_gpu.py where nothing else is said."""
import numpy as np
import pytest
import torch

from tests.test_linattn_gpu import check, make, n64, reference, run
from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0, 5])
def test_no_sequences_give_zero_decay_gradients(gpu, T):
    """A decay per head belongs to no sequence: its gradient over an empty batch is zero, and is written."""
    import scan_linear_rnns_amd as mgs
    say(f"linattn B=0 T={T} decay per head")
    a = make(gpu, 0, T, 3, 1, 32, 48, decay="head")
    outs = (torch.empty(0, T, 1, 32, device=gpu), torch.empty(0, T, 1, 32, device=gpu),
            torch.empty(0, T, 3, 48, device=gpu), torch.full((3,), float("nan"), device=gpu),
            torch.empty(0, 3, 48, 32, device=gpu))
    got = mgs.mgs_linattn_bwd(*(a[n] for n in ("q", "k", "v", "g", "do")), out=outs)
    assert got[3] is outs[3] and torch.equal(got[3], torch.zeros(3, device=gpu))
    assert run(a, 1.0)["dg"].count_nonzero() == 0


def packed(gpu, T, starts, dtype, seed):
    """One sequence of T steps holding documents that begin at `starts` (0 first) with a cleared state."""
    a = make(gpu, 2, T, 2, 1, 64, 64, dtype, S0=True, seed=seed)
    a["g"][:, starts[1:]] = float("-inf")
    return a


def document(a, t0, t1):
    """Its inputs alone: the state it is entered with counts for the first, the last one's gradient for the last."""
    T = a["q"].shape[1]
    cut = {n: a[n][:, t0:t1] for n in ("q", "k", "v", "g", "do")}
    return dict(cut, S0=a["S0"] if t0 == 0 else None, dST=a["dST"] if t1 == T else None, lengths=None)


PACKS = [(200, [0, 1]), (200, [0, 63, 64, 65, 128]), (600, [0, 100, 255, 256, 257, 511]), (1100, [0, 300, 512, 900]),
         (700, [0, 512]), (600, [0, 5, 40, 41, 42, 590])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,starts", PACKS)
def test_cleared_states_part_the_gradients_of_documents(gpu, T, starts, dtype):
    """Across a cleared state nothing reaches the documents before it, rounding errors neither: with each document's
    gradients 10^3 times the one's before it, every one is as good as alone.  (A document may lie across one more
    chunk than it would alone: one of the bound's 240 additions.)"""
    say(f"linattn packed T={T} {starts} {dtype}")
    a = packed(gpu, T, starts, dtype, T + len(starts))
    ends = starts[1:] + [T]
    for i, (t0, t1) in enumerate(zip(starts, ends)):
        a["do"][:, t0:t1] *= 10.0 ** (3 * i)
    a["dST"] *= 10.0 ** (3 * len(starts) - 3)
    got = run(a, 0.125)
    for t0, t1 in zip(starts, ends):
        check({n: got[n][:, t0:t1] for n in ("o", "dq", "dk", "dv", "dg")}, document(a, t0, t1), 0.125, f"{t0}..{t1}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,starts", PACKS)
def test_non_finite_values_stay_out_of_earlier_documents(gpu, T, starts, dtype):
    """A NaN value in the last document's second half (or only step) reaches no output of the documents before it."""
    say(f"linattn packed with NaN T={T} {starts} {dtype}")
    a = packed(gpu, T, starts, dtype, 7 * T + len(starts))
    a["v"][:, (starts[-1] + T) // 2, 1, 5] = float("nan")
    got = run(a, 0.125)
    assert torch.isnan(got["o"][:, T - 1, 1, 5]).all() and torch.isnan(got["ST"][:, 1, 5]).all()
    for t0, t1 in zip(starts[:-1], starts[1:]):
        part = {n: got[n][:, t0:t1] for n in ("o", "dq", "dk", "dv", "dg")}
        check(part, document(a, t0, t1), 0.125, f"{t0}..{t1}")


@pytest.mark.parametrize("B,T,H,d", [(1, 2100, 2, 64), (2, 700, 2, 128), (64, 140, 8, 64), (64, 140, 8, 128), (3, 50, 2, 64)],
                         ids=["segments 64", "segments 128", "one piece 64", "one piece 128", "one chunk"])
def test_outputs_do_not_depend_on_what_else_is_asked_for(gpu, B, T, H, d):
    """o with and without the final state, the gradients with and without dS0, aligned rows or not: the same bits."""
    import scan_linear_rnns_amd as mgs
    say(f"linattn outputs asked for B={B} T={T} H={H} d={d}")
    a = make(gpu, B, T, H, H, d, d, "bf16", seed=T + d)
    ins = [a[n] for n in ("q", "k", "v", "g")]
    o, ST, _ = mgs.mgs_linattn_fwd(*ins, scale=0.1)
    assert torch.equal(mgs.mgs_linattn_fwd(*ins, scale=0.1, want_state=False)[0], o)
    full = mgs.mgs_linattn_bwd(*ins, a["do"], scale=0.1)
    part = [torch.empty_like(t) for t in full[:4]]
    mgs.mgs_linattn_bwd(*ins, a["do"], scale=0.1, out=(*part, None))
    for n, x, y in zip(("dq", "dk", "dv", "dg"), full, part):
        assert torch.equal(x, y), n
    c = dict(a)
    for n in ("q", "k", "v", "do"):
        pad = torch.empty(*a[n].shape[:3], d + 3, dtype=a[n].dtype, device=gpu)
        pad[..., 1:-2] = a[n]
        c[n] = pad[..., 1:-2]
    got = run(c, 0.1)
    for n, y in zip(("o", "ST", "dq", "dk", "dv", "dg", "dS0"), (o, ST, *full)):
        assert torch.equal(got[n], y), n


@pytest.mark.parametrize("per_head", [False, True], ids=["decay per step", "decay per head"])
def test_step_decay_is_an_exponential_of_fp32(gpu, per_head):
    """With k = 0 the state is only scaled, by e^g: the exponential is good to 2^-23 (an ulp), its correction and the
    product are rounded, 2^-24 each.  Cleared states, overflow and NaN are exact."""
    import scan_linear_rnns_amd as mgs
    say("linattn step decays")
    B, H, d = 4, 64, 64
    gen = torch.Generator().manual_seed(41)
    S = torch.randn(B, H, d, d, generator=gen).to(gpu)
    k = torch.zeros(B, 1, d, device=gpu)
    v = torch.randn(B, H, d, generator=gen).to(gpu)
    g = -torch.logspace(-4, 1.9, H).repeat(B, 1).to(gpu)      # to -79.4
    g = g * (1 + 0.1 * torch.rand(B, H, generator=gen)).to(gpu)
    if per_head:
        g = g[0].contiguous()
    want = torch.exp(g.double()).expand(B, H)[..., None, None] * S.double()
    mgs.mgs_linattn_step(k, k, v, g, S)
    assert bool(((S.double() - want).abs() <= 4.01 * 2.0 ** -24 * want.abs() + 2.0 ** -149).all())
    before = S.clone()
    edge = torch.tensor([float("-inf"), -3.0e38, 0.0, -1200.0, 89.0, float("inf"), float("nan"), -0.0], device=gpu)
    g = edge.repeat(8).expand(B, H) if not per_head else edge.repeat(8)
    mgs.mgs_linattn_step(k, k, v, g, S)
    S, before = S.view(B, 8, 8, d, d), before.view(B, 8, 8, d, d)
    for i in (0, 1, 3):
        assert S[:, :, i].count_nonzero() == 0
    for i in (2, 7):
        assert torch.equal(S[:, :, i], before[:, :, i])
    assert torch.isnan(S[:, :, 6]).all()
    assert not torch.isfinite(S[:, :, 5]).any()


def test_step_growth_past_fp32_is_infinite(gpu):
    """Where e^g overflows, a state becomes an infinity of its sign, whatever the exponent's tail is (zero for some)."""
    import scan_linear_rnns_amd as mgs
    say("linattn step growth")
    H, d = 512, 16
    S = torch.randn(1, H, d, d, generator=torch.Generator().manual_seed(43)).to(gpu)
    z = torch.zeros(1, 1, d, device=gpu)
    g = torch.linspace(88.75, 400.0, H, device=gpu)[None]
    g[0, 0], g[0, 1] = 1e30, float("inf")
    want = S.sign() * float("inf")
    mgs.mgs_linattn_step(z, z, torch.zeros(1, H, d, device=gpu), g, S)
    assert torch.equal(S, want)


def check_cut(got, a, scale, who=""):
    """check() where an output in bf16 comes of two bf16 terms: each state and score on its way there is cut to within
    2^-18 of itself (8 bits and 8 of the rest), so the bound of test_linattn_gpu.py grows by 2^-18 of the sum of
    absolute terms.  Everything that is not rounded to bf16 has to meet the bound as it is."""
    want, size = reference(a, scale)
    T, dk, dv = a["q"].shape[1], a["q"].shape[3], a["v"].shape[3]
    gamma = (dk + dv + 64 + -(-T // 64) + 48) * 2.0 ** -24
    for name, t in got.items():
        x = n64(t)
        tol = gamma * size[name]
        if t.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -18 * size[name] + 2.0 ** -8 * np.abs(want[name])
        assert x.shape == want[name].shape, (who, name)
        bad = ~(np.abs(x - want[name]) <= tol)
        assert not bad.any(), (who, name, int(bad.sum()), float(np.abs(x - want[name])[bad].max()))


@pytest.mark.parametrize("B,T,H,d", [(1, 1300, 2, 64), (1, 600, 2, 128), (260, 70, 2, 64), (2, 100, 2, 128)],
                         ids=["segments 64", "segments 128", "one piece 64", "few chunks 128"])
def test_output_alone(gpu, B, T, H, d):
    """The forward of a training step: no final state is asked for."""
    import scan_linear_rnns_amd as mgs
    say(f"linattn output alone B={B} T={T} H={H} d={d}")
    a = make(gpu, B, T, H, H, d, d, "bf16", seed=T, back=False)
    o, ST, _ = mgs.mgs_linattn_fwd(*(a[n] for n in ("q", "k", "v", "g")), scale=d ** -0.5, want_state=False)
    assert ST is None
    check_cut(dict(o=o), a, d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S0", [True, False], ids=["states", "no states"])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_many_walks(gpu, d, S0, dtype):
    """Over 256 (sequence, head, segment) triples: dv's walk is a launch of its own, in reverse, with and without the
    states' gradients."""
    import scan_linear_rnns_amd as mgs
    B, T, H = 33, 70, 8
    say(f"linattn many walks d={d} states={S0} {dtype}")
    a = make(gpu, B, T, H, H, d, d, dtype, S0=S0, seed=d)
    ins = [a[n] for n in ("q", "k", "v", "g")]
    outs = [torch.empty_like(a[n]) for n in ("q", "k", "v")] + [torch.empty_like(a["g"])]
    dS0 = torch.empty(B, H, d, d, device=gpu) if S0 else None
    mgs.mgs_linattn_bwd(*ins, a["do"], S0=a["S0"], dST=a["dST"], scale=d ** -0.5, out=(*outs, dS0))
    got = dict(zip(("dq", "dk", "dv", "dg"), outs))
    if S0:
        got["dS0"] = dS0
    check_cut(got, a, d ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(2, 4, 2, 64, 64), (3, 2, 1, 33, 17), (70, 8, 8, 64, 128)])
def test_step_with_a_decay_per_head(gpu, B, H, Hk, dk, dv, dtype):
    import scan_linear_rnns_amd as mgs
    say(f"linattn step, decay per head B={B} H={H} dk={dk} dv={dv} {dtype}")
    a = make(gpu, B, 1, H, Hk, dk, dv, dtype, decay="head", S0=True, seed=B, back=False)
    want, size = reference(a, 0.3)
    S = a["S0"].clone()
    o = mgs.mgs_linattn_step(a["q"][:, 0], a["k"][:, 0], a["v"][:, 0], a["g"], S, scale=0.3)
    gamma = (dk + 48) * 2.0 ** -24
    assert (np.abs(n64(S) - want["ST"]) <= gamma * size["ST"]).all()
    last = 2.0 ** -8 * np.abs(want["o"][:, 0]) if dtype == "bf16" else 0.0
    assert (np.abs(n64(o) - want["o"][:, 0]) <= gamma * size["o"][:, 0] + last).all()


def test_infinite_values_are_not_finite_from_their_step_on(gpu):
    """An infinity in v makes its column's outputs and state not finite from its step on (NaN or infinite), and
    touches no earlier step and no other column."""
    say("linattn infinite values")
    for dtype in ("f32", "bf16"):
        for value in (float("inf"), float("-inf")):
            a = make(gpu, 1, 200, 1, 1, 64, 64, dtype, back=False, seed=47)
            a["v"][0, 70, 0, 3] = value
            got = run(a, 1.0)
            o = got["o"].float()
            assert torch.isfinite(o[0, :70]).all() and not torch.isfinite(o[0, 70:, 0, 3]).any()
            other = torch.arange(64, device=gpu) != 3
            assert torch.isfinite(o[..., other]).all() and torch.isfinite(got["ST"][:, :, other]).all()
            assert not torch.isfinite(got["ST"][0, 0, 3]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,at", [(200, 70), (1100, 600), (150, 149), (640, 0), (640, 511), (640, 512)])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_non_finite_values_stay_on_their_side(gpu, name, T, at, dtype):
    """A value that is not finite at one step reaches only the outputs whose sums hold it: with q and do their own
    step's o and dq and the earlier steps' dk and dv, with k and v the later steps' o and dq and their own dv and dk;
    and nothing of another head."""
    say(f"linattn non-finite {name} T={T} at={at} {dtype}")
    t = torch.arange(T, device=gpu)
    later, earlier, own, none = t >= at, t <= at, t == at, t < 0
    may = {"q": dict(o=own, dq=none, dk=earlier, dv=earlier), "do": dict(o=none, dq=own, dk=earlier, dv=earlier),
           "k": dict(o=later, dq=later, dk=none, dv=own), "v": dict(o=later, dq=later, dk=own, dv=none)}[name]
    for value in (float("nan"), float("inf")):
        a = make(gpu, 1, T, 2, 2, 64, 64, dtype, S0=True, seed=at)
        a[name][0, at, 0, 5] = value
        got = run(a, 0.1)
        for n, steps in may.items():
            x = got[n].float()
            assert torch.isfinite(x[:, :, 1]).all(), n
            assert bool((torch.isfinite(x[0, :, 0]).all(-1) | steps).all()), n
        assert torch.isfinite(got["dg"][:, :, 1]).all()
