"""GPU parity of the gated linear recurrence (mgs_gated_fwd, _bwd, _step) with its definition in 64 bits.

Tolerances, element by element, are running bounds that the reference carries through the recurrence with the values.
A sigmoid is an exponential (an ulp, its argument's rounding made good for fp32 and 2^-24 |z| off for bf16), a sum and
a reciprocal (an ulp): within 2^-21 of itself, and 2^-23 |z| more in bf16.  log a multiplies by softplus(lam) (two ulps)
and rounds: within eps = 2^-20 (and the bf16 part at the largest |r|).  a is off by |log a| eps and an ulp of the
exponential, sqrt(1 - a^2) by 2 eps (its series and 1 - a^2 keep relative accuracy), b = beta iota x by 4 eps.  Each step
multiplies and adds: 2^-24 of what is held, once in the chunk and once in the pair of the chunk, on both ways, with the
exponential's ulp: eps_step = 2^-22.  1 - a^2 below the smallest normal number, 2^-126, may count as 0: its root is off by
up to 2^-63 besides (2^-62 with what rounds before it).  An output in bf16 is rounded by 2^-8 of itself more."""
import numpy as np
import pytest
import torch

from tests import tokens_reference as ref
from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("y", "hT", "dx", "dr", "di", "dlam", "dh0")


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(dev, B, T, D, dtype="f32", h0=True, dhT=True, lengths=None, reset=0.0, seed=0, fused=False, big=1.0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DT[dtype]
    if fused:
        x, r, i = (big * rand(B, T, 3 * D)).to(dt).to(dev).split(D, dim=2)
    else:
        x, r, i = ((big * rand(B, T, D)).to(dt).to(dev) for _ in range(3))
    a = dict(x=x, r=r, i=i, lam=(rand(D) * 2 - 4).to(dev), h0=rand(B, D).to(dev) if h0 else None,
             dy=rand(B, T, D).to(dt).to(dev), dhT=rand(B, D).to(dev) if dhT else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev),
             reset=(torch.rand(B, T, generator=g) < reset).to(dev) if reset else None)
    return a


def run(a, rate=8.0, ws=None):
    import scan_linear_rnns_amd as mgs
    inputs = (a["x"], a["r"], a["i"], a["lam"])
    more = dict(lengths=a["lengths"], reset=a["reset"], rate=rate, ws=ws)
    y, hT, states = mgs.mgs_gated_fwd(*inputs, h0=a["h0"], want_states=True, **more)
    got = mgs.mgs_gated_bwd(*inputs, a["dy"], states, dhT=a["dhT"], **more)
    return dict(zip(NAMES, (y, hT, *got)))


def reference(a, rate=8.0):
    r = n64(a["r"])
    live = np.abs(r[np.isfinite(r)])
    eps = 2.0 ** -20 + (2.0 ** -23 * live.max(initial=0.0) if a["x"].dtype == torch.bfloat16 else 0.0)
    return ref.gated(*(n64(a[n]) for n in ("x", "r", "i", "lam")), h0=n64(a["h0"]),
                     lengths=None if a["lengths"] is None else a["lengths"].cpu().numpy(),
                     reset=None if a["reset"] is None else a["reset"].cpu().numpy(), rate=rate, dy=n64(a["dy"]),
                     dhT=n64(a["dhT"]), eps=eps, eps_step=2.0 ** -22, tiny=2.0 ** -62)


def check(got, want, names=NAMES, who=""):
    for n in names:
        x, w = n64(got[n]), want[n]
        assert x.shape == w.shape, (who, n)
        tol = want["err"][n] + (2.0 ** -8 if got[n].dtype == torch.bfloat16 else 2.0 ** -24) * np.abs(w) + 1e-37
        bad = ~(np.abs(x - w) <= tol)
        assert not bad.any(), (who, n, int(bad.sum()), np.argwhere(bad)[:3].tolist(), x[bad][:4], w[bad][:4],
                               tol[bad][:4])


LENGTHS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1023, 1024, 1025, 1153]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(gpu, T, dtype):
    say(f"gated T={T} {dtype}")
    a = make(gpu, 2, T, 130, dtype, seed=T)
    check(run(a), reference(a))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 63, 64, 127, 128, 129, 255, 257, 1000])
def test_widths(gpu, D, dtype):
    say(f"gated D={D} {dtype}")
    a = make(gpu, 3, 140, D, dtype, seed=D)
    check(run(a), reference(a))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fused", [False, True])
def test_ragged_packed_and_fused(gpu, dtype, fused):
    """Lengths from none to past T; what lies behind a length is not looked at; documents of a few steps and of many."""
    say(f"gated ragged packed {dtype} fused={fused}")
    for T, reset in ((300, 0.02), (1400, 0.0), (70, 0.5)):
        a = make(gpu, 6, T, 96, dtype, lengths=[0, 1, T - 1, T + 5, -3, T // 2], reset=reset, seed=T, fused=fused)
        want = reference(a)
        for b, n in enumerate((0, 1, T - 1, T, 0, T // 2)):
            for name in ("x", "r", "i", "dy"):
                a[name][b, n:] = float("nan")
            if a["reset"] is not None:
                a["reset"][b, n:] = True
        check(run(a), want)


def test_no_state_in_or_out(gpu):
    import scan_linear_rnns_amd as mgs
    say("gated without states")
    a = make(gpu, 2, 200, 48, h0=False, dhT=False)
    want = reference(a)
    check(run(a), want)
    y, hT, states = mgs.mgs_gated_fwd(a["x"], a["r"], a["i"], a["lam"], want_state=False)
    assert hT is None and states is None
    check(dict(y=y), want, ["y"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_at_their_ends(gpu, dtype):
    """Pre-activations of up to +-60 and decays from none to all of a step's: closed gates hold the state, open ones
    clear it."""
    say(f"gated ends {dtype}")
    a = make(gpu, 2, 150, 64, dtype, seed=5, big=20.0)
    a["lam"] = torch.linspace(-60, 30, 64, device=gpu)
    check(run(a), reference(a))


def test_infinite_preactivations(gpu):
    """r = -inf: the state is held, nothing comes in, and no gradient is NaN; r = +inf, i = +-inf: the limits."""
    say("gated infinite pre-activations")
    a = make(gpu, 1, 100, 8, seed=6)
    a["r"][:, 10:20] = float("-inf")
    a["r"][:, 30] = float("inf")
    a["i"][:, 40] = float("-inf")
    a["i"][:, 50] = float("inf")
    got = run(a)
    for n in NAMES:
        assert torch.isfinite(got[n]).all(), n
    h = got["y"]
    # (a chunk's steps are walked, a later one's state is its pair's product and sum: some 20 roundings of sums below 4)
    assert (h[:, 10:20] - h[:, 9:10]).abs().max() <= 20 * 4 * 2.0 ** -24
    assert got["dr"][:, 10:20].count_nonzero() == 0 and got["di"][:, 40].count_nonzero() == 0
    check(got, reference(a))


@pytest.mark.parametrize("T", [100, 1500])
def test_documents_do_not_see_each_other(gpu, T):
    """What a document holds, finite or not, reaches no later one, and its gradient no earlier one."""
    say(f"gated documents T={T}")
    a = make(gpu, 1, T, 40, seed=7)
    cut = T // 2 + 3
    a["reset"] = torch.zeros(1, T, dtype=torch.uint8, device=gpu)
    a["reset"][0, cut] = 255
    clean = run(a)
    a["h0"][:] = float("inf")
    a["x"][0, cut // 2] = float("nan")
    got = run(a)
    for n in ("y", "dx", "dr", "di"):
        assert torch.equal(got[n][:, cut:], clean[n][:, cut:]), n
    assert torch.equal(got["hT"], clean["hT"]) and not torch.isfinite(got["y"][:, cut - 1]).any()
    b = make(gpu, 1, T, 40, seed=7)
    b["reset"] = a["reset"]
    b["dhT"][:] = float("inf")
    b["dy"][0, cut] = float("nan")
    got = run(b)
    for n in ("y", "dx", "dr", "di"):
        assert torch.equal(got[n][:, :cut], clean[n][:, :cut]), n
    assert torch.equal(got["dh0"], clean["dh0"])


def test_non_finite_values_stay_in_their_channel(gpu):
    say("gated NaN")
    a = make(gpu, 2, 700, 70, seed=8)
    clean = run(a)
    a["x"][1, 300, 17] = float("nan")
    a["r"][0, 5, 69] = float("nan")
    got = run(a)
    other = torch.ones(70, dtype=torch.bool, device=gpu)
    other[[17, 69]] = False
    for n in NAMES:
        assert torch.equal(got[n][..., other], clean[n][..., other]), n
    assert torch.isnan(got["y"][1, 300:, 17]).all() and torch.equal(got["y"][1, :300], clean["y"][1, :300])
    assert torch.isnan(got["y"][0, 5:, 69]).all() and torch.isnan(got["dlam"][[17, 69]]).all()


def test_halves_joined_by_their_state(gpu):
    """A sequence in two calls: the second from the first's state, the gradient back through it."""
    import scan_linear_rnns_amd as mgs
    say("gated halves")
    a = make(gpu, 2, 400, 64, seed=9)
    want, cut = reference(a), 171
    parts = [{k: (v[:, s] if k in ("x", "r", "i", "dy") else v) for k, v in a.items()}
             for s in (slice(0, cut), slice(cut, None))]
    parts[1]["h0"] = mgs.mgs_gated_fwd(*(parts[0][n] for n in ("x", "r", "i", "lam")), h0=a["h0"])[1]
    late = run(parts[1])
    parts[0]["dhT"] = late["dh0"]
    early = run(parts[0])
    got = {n: torch.cat([early[n], late[n]], 1) for n in ("y", "dx", "dr", "di")}
    got.update(hT=late["hT"], dh0=early["dh0"], dlam=early["dlam"] + late["dlam"])
    check(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 64, 77, 513, 2048])
def test_step(gpu, D, dtype):
    """A step is the sequence's first; slots in no order; idle ones give zeros and touch nothing."""
    import scan_linear_rnns_amd as mgs
    say(f"gated step D={D} {dtype}")
    a = make(gpu, 5, 1, D, dtype, seed=D)
    want = reference(a)
    slots = torch.tensor([7, 0, -1, 3, 9], dtype=torch.int32, device=gpu)
    h = torch.full((9, D), 5.0, device=gpu)
    for b in (0, 1, 3):
        h[slots[b].long()] = a["h0"][b]
    y = mgs.mgs_gated_step(a["x"][:, 0], a["r"][:, 0], a["i"][:, 0], a["lam"], h, slots=slots)
    for b in (0, 1, 3):
        err = want["err"]
        one = {"y": want["y"][b], "hT": want["hT"][b:b + 1], "err": {"y": err["y"][b], "hT": err["hT"][b:b + 1]}}
        check(dict(y=y[b:b + 1], hT=h[slots[b].long()][None]), one, ["y", "hT"])
    assert y[[2, 4]].count_nonzero() == 0 and (h[[1, 2, 4, 5, 6, 8]] == 5.0).all()
    h = a["h0"].clone()
    y2 = mgs.mgs_gated_step(a["x"][:, 0], a["r"][:, 0], a["i"][:, 0], a["lam"], h)
    assert torch.equal(y2[[0, 1, 3]], y[[0, 1, 3]])


def test_steps_are_the_sequence(gpu):
    import scan_linear_rnns_amd as mgs
    say("gated steps")
    a = make(gpu, 3, 40, 96, seed=11, fused=True)
    h, rows = a["h0"].clone(), []
    for t in range(40):
        rows.append(mgs.mgs_gated_step(a["x"][:, t], a["r"][:, t], a["i"][:, t], a["lam"], h))
    want = reference(a)
    check(dict(y=torch.stack(rows, 1), hT=h), want, ["y", "hT"])


def test_same_bits_every_time_on_one_workspace(gpu):
    """Across calls of other sizes and types on the same workspace too."""
    import scan_linear_rnns_amd as mgs
    say("gated determinism")
    sizes = [(2, 3000, 300, "f32"), (1, 700, 64, "bf16"), (5, 1300, 130, "bf16"), (3, 64, 64, "f32")]
    args = [make(gpu, *s, seed=i, reset=0.01) for i, s in enumerate(sizes)]
    ones = [run(a) for a in args]
    ws = mgs.workspace(max(mgs.mgs_gated_workspace_size(*s[:3], dtype=DT[s[3]], backward=True) for s in sizes), gpu)
    for _ in range(6):
        for a, one in zip(args, ones):
            got = run(a, ws=ws)
            for n in NAMES:
                assert torch.equal(got[n], one[n]), n
    assert mgs.mgs_workspace_check(ws) == 0


def test_strided_and_odd_aligned_inputs_give_the_same_bits(gpu):
    say("gated strides")
    for dt in ("f32", "bf16"):
        a = make(gpu, 2, 200, 64, dt, seed=12)
        one = run(a)
        b = dict(a)
        for n in ("x", "r", "i", "dy"):
            raw = torch.empty(2, 210, 67, dtype=DT[dt], device=gpu)
            raw[:, 10:, 3:] = a[n]
            b[n] = raw[:, 10:, 3:]
        got = run(b)
        for n in NAMES:
            assert torch.equal(got[n], one[n]), n
        c = dict(a, x=a["x"][:, :1].expand(2, 200, 64))   # one row for all steps
        d = dict(a, x=c["x"].contiguous())
        got, one = run(c), run(d)
        for n in NAMES:
            assert torch.equal(got[n], one[n]), n


def test_waits_give_up_and_recover(gpu):
    import scan_linear_rnns_amd as mgs
    say("gated failure path")
    a = make(gpu, 2, 3000, 256, seed=13)
    ws = mgs.workspace(mgs.mgs_gated_workspace_size(2, 3000, 256, backward=True), gpu)
    one = run(a, ws=ws)
    mgs.mgs_workspace_set_waits(ws, spin_limit=4, fail_waits=True)
    run(a, ws=ws)
    torch.cuda.synchronize()
    assert mgs.mgs_workspace_check(ws) & 1
    mgs.mgs_workspace_set_waits(ws, 0, False)
    got = run(a, ws=ws)
    for n in NAMES:
        assert torch.equal(got[n], one[n]), n
    assert mgs.mgs_workspace_check(ws) == 0


def test_empty_batch(gpu):
    say("gated empty batch")
    for T in (0, 5):
        a = make(gpu, 0, T, 9, seed=14)
        got = run(a)
        assert got["dlam"].shape == (9,) and got["dlam"].count_nonzero() == 0


def test_step_of_more_channels_than_bytes_fit_32_bits(gpu):
    """2^30 and some channels of four bytes: the ends and the 32-bit seam are what those channels give alone."""
    import gc
    import scan_linear_rnns_amd as mgs
    D = (1 << 30) + 10
    say(f"gated step D={D}")
    g = torch.Generator(gpu).manual_seed(1)
    rand = lambda n: torch.randn(n, D, generator=g, device=gpu)  # noqa: E731
    x, r, i, h, lam = rand(1), rand(1), rand(1), rand(1), rand(1)[0].sub_(4)
    at = torch.tensor([0, 1, 511, 512, (1 << 29) - 1, 1 << 29, (1 << 30) - 1, 1 << 30, D - 2, D - 1], device=gpu)
    small = h[:, at].clone()
    want = mgs.mgs_gated_step(*(t[:, at].contiguous() for t in (x, r, i)), lam[at].contiguous(), small)
    y = mgs.mgs_gated_step(x, r, i, lam, h)
    assert torch.equal(y[:, at], want) and torch.equal(h[:, at], small)
    del x, r, i, h, lam, y
    gc.collect()
    torch.cuda.empty_cache()


def test_far_offsets(gpu):
    """Rows whose strides put them past 2^32 bytes from the first."""
    say("gated far rows")
    a = make(gpu, 2, 70, 128, "bf16", seed=15)
    one = run(a)
    b = dict(a)
    room = torch.empty((1 << 31) + 70 * 130, dtype=torch.bfloat16, device=gpu)
    b["x"] = room.as_strided((2, 70, 128), (1 << 31, 130, 1))
    b["x"].copy_(a["x"])
    got = run(b)
    for n in NAMES:
        assert torch.equal(got[n], one[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [9, 200])
def test_many_short_sequences(gpu, T, dtype):
    say(f"gated 40 x {T} {dtype}")
    a = make(gpu, 40, T, 70, dtype, lengths=[(7 * b) % (T + 1) for b in range(40)], reset=0.1, seed=T)
    check(run(a), reference(a))
