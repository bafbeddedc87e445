"""GPU parity of sampling (mgs_sample) with its definition in 64 bits: tokens are equal wherever the reference's
decisions are more than 2^-36 of the weight from the next other one (weights are within 2^-43 of the largest, and sums
of up to 2^17 of them are compared here); logp is the log of a share that close, rounded to fp32: 2^-24 |logp| + 2^-23."""
import numpy as np
import pytest
import torch

from tests import tokens_reference as ref
from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def settings(B, seed, **fixed):
    rng = np.random.default_rng(seed)
    s = dict(temperature=rng.uniform(0.3, 1.5, B).astype(np.float32), top_k=rng.integers(0, 300, B).astype(np.int32),
             top_p=rng.uniform(0.2, 1.1, B).astype(np.float32), min_p=rng.uniform(-0.05, 0.2, B).astype(np.float32))
    for k, v in fixed.items():
        s[k] = np.full(B, v, s[k].dtype)
    return s


def check(logits, u, s, token, logp, who=""):
    x, u, token, logp = (t.detach().double().cpu().numpy() for t in (logits, u, token, logp))
    close = 0
    for b in range(len(u)):
        want, lp, margin = ref.sample(x[b], float(u[b]), float(s["temperature"][b]), int(s["top_k"][b]),
                                      float(s["top_p"][b]), float(s["min_p"][b]))
        if margin < 2.0 ** -36:
            close += 1
            continue
        assert token[b] == want, (who, b, token[b], want, margin, {k: v[b] for k, v in s.items()})
        assert logp[b] == lp or abs(logp[b] - lp) <= 2.0 ** -24 * abs(lp) + 2.0 ** -23, (who, b, logp[b], lp)
    assert close <= len(u) // 10, (who, close)


def draw(dev, B, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(B, V, generator=g)
    x = x.masked_fill(torch.rand(B, V, generator=g) < 0.05, float("-inf"))
    x[:, V // 2] = 1.0   # (a row has a token)
    return x.to(DT[dtype]).to(dev), torch.rand(B, generator=g).to(dev)


def run(logits, u, s):
    import scan_linear_rnns_amd as mgs
    dev = u.device
    return mgs.mgs_sample(logits, u, **{k: torch.from_numpy(v).to(dev) for k, v in s.items()})


VOCABS = [1, 2, 3, 63, 64, 65, 500, 1023, 1025, 4096, 5003, 32000, 50001, 131072]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
def test_vocabularies(gpu, V, dtype):
    """Every filter alone, all of them, and none."""
    B = 12 if V < 10000 else 6
    say(f"sample V={V} {dtype}")
    x, u = draw(gpu, B, V, dtype, V)
    off = dict(top_k=0, top_p=1.0, min_p=0.0)
    for i, fixed in enumerate([off, dict(top_p=1.0, min_p=0.0), dict(top_k=0, min_p=0.0), dict(top_k=0, top_p=1.0), {}]):
        s = settings(B, V + i, **fixed)
        check(x, u, s, *run(x, u, s), who=fixed)


@pytest.mark.parametrize("B", [1, 2, 37, 256, 700])
def test_batches(gpu, B):
    say(f"sample B={B}")
    x, u = draw(gpu, B, 1500, "f32", B)
    s = settings(B, B)
    token, logp = run(x, u, s)
    check(x, u, s, token, logp)
    # a row's answer does not depend on the batch
    for b in {0, B // 2, B - 1}:
        one = run(x[b:b + 1], u[b:b + 1], {k: v[b:b + 1] for k, v in s.items()})
        assert one[0][0] == token[b] and one[1][0] == logp[b]


def test_numbers_for_all_rows(gpu):
    import scan_linear_rnns_amd as mgs
    say("sample numbers")
    x, u = draw(gpu, 9, 800, "f32", 1)
    for fixed in (dict(), dict(temperature=0.7), dict(top_k=5), dict(top_p=0.8), dict(min_p=0.1),
                  dict(temperature=0.9, top_k=40, top_p=0.9, min_p=0.05), dict(temperature=0.0), dict(top_k=10 ** 9)):
        full = dict(dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **fixed)
        check(x, u, settings(9, 0, **dict(full, top_k=min(full["top_k"], 2 ** 31 - 1))), *mgs.mgs_sample(x, u, **fixed))


@pytest.mark.parametrize("B, V", [(3, 800), (2, 32000), (2, 50001), (2, 200000), (130, 40000), (70, 200000)])
def test_numbers_for_all_rows_bf16(gpu, B, V):
    """(Other kernels than a tensor of settings takes.)"""
    import scan_linear_rnns_amd as mgs
    say(f"sample numbers bf16 {B} x {V}")
    x, u = draw(gpu, B, V, "bf16", V)
    for fixed in (dict(), dict(top_k=5), dict(top_k=700), dict(top_p=0.8), dict(min_p=0.1),
                  dict(temperature=0.9, top_k=40, top_p=0.9, min_p=0.05), dict(temperature=0.0)):
        full = dict(dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **fixed)
        rows = slice(0, min(B, 6))
        token, logp = mgs.mgs_sample(x, u, **fixed)
        check(x[rows], u[rows], settings(B, 0, **full), token[rows], logp[rows], who=fixed)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 70, 5000, 40000, 150000])
def test_no_filters(gpu, V, dtype):
    """Whole rows and cut ones; a largest logit at the end, far ahead of the others, infinite; rows with none."""
    import scan_linear_rnns_amd as mgs
    say(f"sample without filters V={V} {dtype}")
    inf, nan = float("inf"), float("nan")
    x, _ = draw(gpu, 12, V, dtype, V)
    x[1, V - 1] = 200.0
    x[2, :V // 2] = 1000.0
    x[2, 0] = -1000.0
    x[3] = torch.linspace(-3000, 3000, V, device=gpu)
    x[4] = -inf
    x[5, V // 3] = nan
    x[6, V // 2] = x[6, 0] = inf
    x[7] = -inf
    x[7, V - 1] = -5.0
    x[8] = 0.0
    temperature = torch.tensor([1.0, 0.5, 1.0, 2.0, 1.0, 1.0, 1.0, 0.7, 1.0, 0.0, 1e-30, inf], device=gpu)
    s = settings(12, 0, top_k=0, top_p=1.0, min_p=0.0)
    s["temperature"] = temperature.cpu().numpy()
    for value in (0.0, 1e-9, 0.37, 0.9999999):
        u = torch.full((12,), value, device=gpu)
        check(x, u, s, *mgs.mgs_sample(x, u, temperature=temperature), who=value)


def test_bf16_values_that_are_rare(gpu):
    """Near 0 (many of them, filters that end among them), 2^10 and more, -2^10 and less at temperatures where that has
    weight, the lowest number as a mask, infinities and NaN."""
    say("sample rare bf16")
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(12)
    for V in (600, 40000):
        base = torch.randn(14, V, generator=g)
        rows = base.clone()
        rows[0, ::3] = 0.0
        rows[1] = -rows[1].abs()
        rows[1, 5:40] = 2.0 ** -15 * torch.randn(35, generator=g)     # the largest are near 0
        rows[2] = 2.0 ** -14 * rows[2]
        rows[3] = 1e-30 * rows[3]
        rows[4] = 400 * rows[4]
        rows[5] = 2000 + rows[5]
        rows[6] = -3000 + 16 * rows[6]
        rows[7, 7:] = torch.finfo(torch.bfloat16).min
        rows[8, :V - 3] = -1024.0
        rows[8, V - 3:] = 1.0
        rows[9, 3] = inf
        rows[10, V - 1] = nan
        rows[11] = torch.where(rows[11] > 0, -0.0, 0.0)
        rows[12] = rows[12].clamp(max=2.0 ** -20)
        rows[13, :] = -2.0 ** -13
        rows[13, 9] = 2.0 ** -13
        x, u = rows.bfloat16().to(gpu), torch.rand(14, generator=g).to(gpu)
        for i, fixed in enumerate([dict(top_k=0, min_p=0.0), dict(top_p=1.0, min_p=0.0), dict(min_p=0.0),
                                   dict(temperature=1e4, top_k=0), dict(temperature=1e-3), dict(temperature=0.0), {}]):
            s = settings(14, i, **fixed)
            if i == 1:
                s["top_k"][:] = [7, 20, 40, 2, 9, 3, 5, 8, 2, 1, 4, V // 2, V // 2 + 17, 3]
            if i == 2:
                s["top_k"][:] = V - 5
            check(x, u, s, *run(x, u, s), who=(V, i))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties(gpu, dtype):
    """Equal logits by the thousand: of equals the first by index stay."""
    say(f"sample ties {dtype}")
    g = torch.Generator().manual_seed(3)
    for V in (64, 5000, 40000):
        x = torch.randint(0, 4, (40, V), generator=g).float()
        x[:4] = 0.0
        x[4:8] = torch.where(torch.rand(4, V, generator=g) < 0.5, 0.0, -0.0)
        x = x.to(DT[dtype]).to(gpu)
        u = torch.rand(40, generator=g).to(gpu)
        for i, fixed in enumerate([dict(top_p=1.0, min_p=0.0), dict(top_k=0, min_p=0.0), {}]):
            s = settings(40, i, **fixed)
            s["top_k"][:] = s["top_k"] * (V // 300 + 1)
            check(x, u, s, *run(x, u, s), who=(V, fixed))


def test_ends_of_the_settings(gpu):
    say("sample settings' ends")
    x, u = draw(gpu, 1, 700, "f32", 4)
    x, u = x.repeat(16, 1), torch.linspace(0, 0.9999, 16, device=gpu)
    inf, nan = float("inf"), float("nan")
    for fixed in (dict(temperature=1e-30), dict(temperature=1e-42), dict(temperature=1e30), dict(temperature=inf),
                  dict(temperature=-1.0), dict(temperature=nan), dict(top_k=1), dict(top_k=-5), dict(top_k=700),
                  dict(top_k=10000), dict(top_p=0.0), dict(top_p=-1.0), dict(top_p=1e-20), dict(top_p=0.99999994),
                  dict(top_p=nan), dict(top_p=inf), dict(min_p=1.0), dict(min_p=2.0), dict(min_p=nan), dict(min_p=1e-30)):
        full = dict(dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **fixed)
        s = settings(16, 0, **full)
        check(x, u, s, *run(x, u, s), who=fixed)
    s = settings(5, 0, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    u = torch.tensor([-1.0, nan, 1.0, 7.0, inf], device=gpu)
    check(x[:5], u, s, *run(x[:5], u, s), who="u")


def test_rows_without_a_distribution(gpu):
    """Nothing but -inf, NaN anywhere: -1; +inf takes all; a row with one token takes it."""
    say("sample masked rows")
    inf, nan = float("inf"), float("nan")
    for V in (7, 3000, 60000):
        x = torch.randn(8, V, generator=torch.Generator().manual_seed(V))
        x[0] = -inf
        x[1, V - 1] = nan
        x[2, [1, V - 2]] = inf
        x[3] = -inf
        x[3, V - 1] = -3e38
        x[4, :3] = inf
        x[4, 5] = nan
        x[5] = 3e38
        x[6, 0] = -nan
        x, u = x.to(gpu), torch.linspace(0.05, 0.95, 8, device=gpu)
        for fixed in (dict(top_k=0, top_p=1.0, min_p=0.0), dict(temperature=0.0), {}):
            s = settings(8, 1, **fixed)
            token, logp = run(x, u, s)
            check(x, u, s, token, logp, who=(V, fixed))
            assert token[[0, 1, 4, 6]].eq(-1).all() and logp[[0, 1, 4, 6]].eq(-inf).all() and token[3] == V - 1


def test_far_tails(gpu):
    """Weights down to nothing: a spread of thousands, and a field of equal small weights that hold most of the sum."""
    say("sample tails")
    g = torch.Generator().manual_seed(5)
    x = 300 * torch.randn(16, 3000, generator=g)
    y = torch.full((16, 60000), -6.0) + 0.01 * torch.randn(16, 60000, generator=g)
    y[:, 77] = 0.0
    u = torch.rand(16, generator=g).to(gpu)
    for logits in (x.to(gpu), y.to(gpu)):
        for i, fixed in enumerate([dict(top_k=0, top_p=1.0, min_p=0.0), dict(top_k=0, min_p=0.0), {}]):
            s = settings(16, i, **fixed)
            check(logits, u, s, *run(logits, u, s), who=fixed)


def test_neighbouring_numbers_and_small_temperatures(gpu):
    """Logits one or two roundings below the largest, at temperatures that put them around 2^-1000 of its weight."""
    say("sample neighbours")
    for top in (10.0, 1.0, -3.0, 2.0 ** -20, 5e30):
        x = np.full(300, top, np.float32)
        for i in range(1, 300):
            x[i] = np.nextafter(x[i - 1] if i < 4 else x[3], np.float32(-np.inf))
        step = float(x[0]) - float(x[1])
        for k in (0.3, 0.5001, 0.75, 0.999, 1.4, 1.5001, 1.9, 2.6, 700.0):   # steps to 2^-1000
            logits = torch.from_numpy(np.tile(x[::-1].copy(), (8, 1))).to(gpu)
            u = torch.linspace(0, 0.9999, 8, device=gpu)
            for fixed in (dict(), dict(top_k=3), dict(top_p=0.7), dict(min_p=0.5)):
                full = dict(dict(temperature=k * step * 1.4426950408889634 / 1000, top_k=0, top_p=1.0, min_p=0.0), **fixed)
                s = settings(8, 0, **full)
                check(logits, u, s, *run(logits, u, s), who=(top, k, fixed))


def test_logits_over_the_whole_range(gpu):
    """Distances past the largest number, at temperatures that large: their weights are not small."""
    say("sample whole range")
    g = torch.Generator().manual_seed(11)
    for V in (500, 20000):
        x = (6.6e38 * (torch.rand(12, V, generator=g, dtype=torch.float64) - 0.5)).float()
        x[:, :40] = -3.4e38
        x[::2, 40:43] = 3.4e38
        x, u = x.to(gpu), torch.rand(12, generator=g).to(gpu)
        for tau in (1e36, 1e38, 3e38, float("inf")):
            for i, fixed in enumerate([dict(top_k=0, top_p=1.0), dict(top_k=0, min_p=0.0), dict(min_p=0.0)]):
                s = settings(12, i, temperature=tau, **fixed)
                check(x, u, s, *run(x, u, s), who=(V, tau, fixed))


def test_a_small_weight_ahead_of_all_others(gpu):
    """u = 0 takes the first token with any weight, here one near 0, alone in its part of the row."""
    say("sample first weight")
    for dt in ("f32", "bf16"):
        for V in (3000, 90000):
            x = torch.full((3, V), float("-inf"))
            x[:, 5] = torch.tensor([0.0, 1e-20, -2.0 ** -14])
            x[:, V - 400:] = 60.0
            x, u = x.to(DT[dt]).to(gpu), torch.zeros(3, device=gpu)
            s = settings(3, 0, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
            token, logp = run(x, u, s)
            check(x, u, s, token, logp)
            assert (token == 5).all()


def test_strides(gpu):
    """Rows apart, a vocabulary inside a padded one, rows that no wide access can take."""
    say("sample strides")
    for dt in ("f32", "bf16"):
        x, u = draw(gpu, 20, 3003, dt, 6)
        s = settings(20, 6)
        raw = torch.full((20, 3100), float("nan"), dtype=DT[dt], device=gpu)
        for off in (0, 1, 8, 90):
            raw.fill_(float("nan"))
            raw[:, off:off + 3003] = x
            token, logp = run(raw[:, off:off + 3003], u, s)
            want = run(x, u, s)
            assert torch.equal(token, want[0]) and torch.equal(logp, want[1])


def test_shares(gpu):
    """Over many numbers u, evenly spread, each token's count is its share of the weight to within one."""
    import scan_linear_rnns_amd as mgs
    say("sample shares")
    x = torch.tensor([0.3, -1.0, 2.0, 0.0, float("-inf"), 1.0], device=gpu)
    n = 20000
    token, _ = mgs.mgs_sample(x.expand(n, 6), (torch.arange(n, device=gpu) + 0.5) / n)
    want = torch.softmax(x.double(), 0) * n
    assert (torch.bincount(token, minlength=6) - want).abs().max() <= 1.01


def test_empty_batch(gpu):
    import scan_linear_rnns_amd as mgs
    token, logp = mgs.mgs_sample(torch.empty(0, 10, device=gpu), torch.empty(0, device=gpu))
    assert token.shape == logp.shape == (0,)


def test_the_largest_batch(gpu):
    import scan_linear_rnns_amd as mgs
    B, V = (1 << 22) - 1, 5
    say(f"sample B={B}")
    g = torch.Generator(gpu).manual_seed(9)
    x, u = torch.randn(B, V, generator=g, device=gpu), torch.rand(B, generator=g, device=gpu)
    token, logp = mgs.mgs_sample(x, u, top_k=3)
    at = torch.tensor([0, 1, 255, 256, B // 2, B - 2, B - 1], device=gpu)
    one = mgs.mgs_sample(x[at], u[at], top_k=3)
    assert torch.equal(token[at], one[0]) and torch.equal(logp[at], one[1])
    assert int(token.min()) >= 0 and int(token.max()) < V and bool((logp <= 0).all())


def test_the_largest_vocabulary(gpu):
    say("sample vocabulary of 2^20")
    for B in (1, 3):
        x, u = draw(gpu, B, 1 << 20, "bf16", B)
        for i, fixed in enumerate([dict(top_k=0, top_p=1.0, min_p=0.0), dict(top_k=0, min_p=0.0), {}]):
            s = settings(B, i, **fixed)
            check(x, u, s, *run(x, u, s), who=fixed)
