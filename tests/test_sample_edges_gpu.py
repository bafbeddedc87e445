"""Where sampling (mgs_sample) can go wrong beside what test_sample_gpu.py covers: values above a row's largest at small
temperatures, and top-p's end in the multiples of 2^-43 that the header states."""
from fractions import Fraction
from math import ceil

import numpy as np
import pytest
import torch

from tests.test_parity_gpu import say
from tests.test_sample_gpu import check, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tau, top", [(1.59e-14, -100.0), (2.45e-18, -100.0), (1e-12, -2.0), (3.7e-26, 0.5)])
def test_small_temperatures_of_counted_rows(gpu, tau, top):
    """A value above the largest has no weight there, whatever e^(distance / temperature) would be: with the first two
    settings a 2^1024 of one value."""
    import scan_linear_rnns_amd as mgs
    say(f"sample counted, temperature {tau}")
    V = 3001
    x = top - 4.0 * torch.rand(6, V, generator=torch.Generator().manual_seed(1)).abs()
    x[:, [V - 1, 1700]] = top
    x = x.bfloat16().to(gpu)
    u = torch.tensor([0.0, 0.2, 0.49, 0.51, 0.8, 0.999], device=gpu)
    for fixed in (dict(top_p=0.9), dict(top_p=0.4), dict(top_k=600, top_p=0.9), dict(top_k=600, min_p=0.5)):
        full = dict(dict(temperature=tau, top_k=0, top_p=1.0, min_p=0.0), **fixed)
        token, logp = (torch.full((6,), -7, dtype=t, device=gpu) for t in (torch.int64, torch.float32))
        mgs.mgs_sample(x, u, **full, token=token, logp=logp)
        check(x, u, settings(6, 0, **full), token, logp, who=fixed)


def by_multiples(x, u, top_k, top_p):
    """(token, logp) of a row at temperature 1 where top-p compares the weights rounded to multiples of 2^-43."""
    x = np.asarray(x, np.float64)
    w = np.exp(x - x.max())
    order = np.argsort(-x, kind="stable")
    if top_k > 0:
        order = order[:top_k]
    q = np.rint(w[order] * 2.0 ** 43).astype(np.int64)
    ahead = np.cumsum(q) - q
    want = max(1, ceil(Fraction(float(np.float32(top_p))) * int(q.sum())))
    ids = np.sort(order[ahead < want])
    run = np.cumsum(w[ids])
    at = int((run <= u * run[-1]).sum())
    return int(ids[at]), float(np.log(w[ids[at]] / run[-1]))


def same(token, logp, want, who):
    assert int(token) == want[0], (who, int(token), want)
    assert abs(float(logp) - want[1]) <= 2.0 ** -24 * abs(want[1]) + 2.0 ** -23, (who, float(logp), want)


@pytest.mark.parametrize("dtype, B", [(torch.float32, 1), (torch.float32, 130), (torch.bfloat16, 1), (torch.bfloat16, 64)])
def test_top_p_ends_in_a_field_of_tiny_weights(gpu, dtype, B):
    """All but one token weigh 0.64 times 2^-43, one step where top-p compares: half of them are kept by the largest
    top_p below 1 (of the weights themselves it would be a quarter; of weights compared with steps, four fifths)."""
    import scan_linear_rnns_amd as mgs
    say(f"sample tiny weights {dtype} B={B}")
    V = 1 << 20
    row = torch.full((V,), -30.25)
    row[V - 1] = 0.0
    x = row.to(dtype).to(gpu).expand(B, V)
    for top_k in (0, V - 5):
        for share in (0.3, 0.5, 0.72):   # of 2^-24: the kept ones hold 0.64 of that
            u = float(np.float32(share * 2.0 ** -24))
            token, logp = mgs.mgs_sample(x, torch.full((B,), u, device=gpu), top_k=top_k, top_p=0.99999994)
            want = by_multiples(row, u, top_k, 0.99999994)
            for b in {0, B - 1}:
                same(token[b], logp[b], want, (top_k, share, b))


# Rows of three logits for which 2^-43's multiples end top-p (a share near that of the first one or two) elsewhere than
# 64-bit weights do: top_p times the sum is a fifth of a step or more from the deciding weight on either side
THREE = [(3, -0.00803716015, -2.61609435, 0.484242082), (3, -0.00227771816, -2.0928452, 0.47146225),
         (3, -0.0132342903, -1.87472475, 0.467235118), (0, -0.00210684282, -0.0105585232, 0.668775678),
         (0, -0.00217477302, -0.0129938666, 0.669307411), (0, -0.00421557622, -0.0108519839, 0.668607473)]


@pytest.mark.parametrize("top_k, second, third, top_p", THREE)
def test_top_p_compares_multiples(gpu, top_k, second, third, top_p):
    """In a short row and in one that is cut into slices; of more logits, the others forbidden."""
    import scan_linear_rnns_amd as mgs
    say(f"sample multiples {top_p}")
    u = torch.tensor([0.999], device=gpu)
    for V in (4, 100000):
        x = torch.full((1, V), float("-inf"))
        x[0, [0, V // 2, V - 1]] = torch.tensor([0.0, second, third])
        token, logp = mgs.mgs_sample(x.to(gpu), u, top_k=top_k, top_p=top_p)
        same(token, logp, by_multiples(x[0], float(u), top_k, top_p), V)


def test_numbers_past_their_types_range(gpu):
    """They count as the nearest number that the type holds."""
    import scan_linear_rnns_amd as mgs
    say("sample numbers past the range")
    inf = float("inf")
    x = torch.randn(40, 300, generator=torch.Generator().manual_seed(2)).to(gpu)
    u = torch.linspace(0, 0.999, 40, device=gpu)
    for given, meant in ((dict(top_k=-2 ** 40), dict()), (dict(top_k=2 ** 40), dict()), (dict(temperature=1e39), dict(temperature=inf)),
                         (dict(temperature=-1e39), dict(temperature=0.0)), (dict(top_p=1e39), dict()),
                         (dict(min_p=1e39), dict(min_p=1.0)), (dict(min_p=-1e39), dict())):
        for got, want in zip(mgs.mgs_sample(x, u, **given), mgs.mgs_sample(x, u, **meant)):
            assert torch.equal(got, want), given


# Rows of which a wave reads its share in several rounds: whole rows, rows cut in two slices, and bf16 rows long enough to
# be counted without a filter.  (B, V, type, places of a round, of a share)
LONG = [(130, 40000, torch.float32, 1024, 2560), (100, 200000, torch.float32, 1024, 6400),
        (130, 70001, torch.bfloat16, 2048, 4608)]


@pytest.mark.parametrize("B, V, dtype, step, share", LONG)
def test_shares_read_in_rounds(gpu, B, V, dtype, step, share):
    """The largest logit, a NaN and an infinity in a share's later rounds, behind smaller ones and ahead of them; numbers
    for all rows, each filter alone and together; a temperature of 0 for some."""
    import scan_linear_rnns_amd as mgs
    say(f"sample rounds {B} x {V} {dtype}")
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(V)
    x = 2.0 * torch.randn(B, V, generator=g)
    late = 3 * share + step + 77   # in the second round of a share
    x[0, late] = 30.0
    x[1, late:late + 3] = torch.tensor([9.0, 25.0, 9.5])
    x[2, :late] -= 40.0
    x[3, :step] = -inf
    x[4, late] = nan
    x[5, late + 5] = inf
    x[6, :] = -inf
    x[6, late + 9] = -7.0
    x[7] = torch.linspace(-60, 60, V)     # each round's largest is larger
    x[8] = torch.linspace(60, -60, V)
    x[9, V - 1] = 20.0
    x = x.to(dtype).to(gpu)
    u = torch.rand(B, generator=g)
    u[:4] = torch.tensor([0.0, 0.4, 0.99999, 0.5])
    u = u.to(gpu)
    rows = slice(0, 14)
    for fixed in (dict(), dict(top_k=5), dict(top_k=700), dict(top_p=0.8), dict(min_p=0.1), dict(temperature=0.0),
                  dict(temperature=0.9, top_k=40, top_p=0.9, min_p=0.05), dict(temperature=30.0)):
        full = dict(dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **fixed)
        token, logp = mgs.mgs_sample(x, u, **fixed)
        check(x[rows], u[rows], settings(14, 0, **full), token[rows], logp[rows], who=fixed)
    # temperatures of their own, without filters: a largest one of 0 in a share's later rounds too
    s = settings(B, 3, top_k=0, top_p=1.0, min_p=0.0)
    s["temperature"][[0, 7, 10]] = 0.0
    s["temperature"][[8, 11]] = np.inf
    token, logp = mgs.mgs_sample(x, u, temperature=torch.from_numpy(s["temperature"]).to(gpu))
    check(x[rows], u[rows], {k: v[rows] for k, v in s.items()}, token[rows], logp[rows], who="own temperatures")
    for i, fixed in enumerate([dict(top_k=0, min_p=0.0), dict(top_p=1.0, min_p=0.0), {}]):
        s = settings(B, i, **fixed)
        token, logp = mgs.mgs_sample(x, u, **{k: torch.from_numpy(v).to(gpu) for k, v in s.items()})
        check(x[rows], u[rows], {k: v[rows] for k, v in s.items()}, token[rows], logp[rows], who=("own", fixed))
