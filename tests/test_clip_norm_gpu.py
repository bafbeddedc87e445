"""GPU parity of the global gradient norm and clipping (mgs_clip_norm) with the sums in 64 bits.

Tolerance: a square is off by at most 2^-24 of itself, and so is the fp32 sum of 8 of them per addition; beyond that
the sums are fp64.  The norm: half of 9 2^-24, and its own rounding, 2^-24: 6 2^-24.  A scaled value: the coefficient's
error (the norm's and two roundings) and its own rounding, 9 2^-24, or 2^-8 more in bf16.
"""
import math

import pytest
import torch

from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def tensors(dev, sizes, dtypes=(torch.float32,), seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(0.1 * (1 + i % 3) * torch.randn(n, generator=g)).to(dtypes[i % len(dtypes)]).to(dev)
            for i, n in enumerate(sizes)]


def check(ts, norm, outs, max_norm):
    n = math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))
    assert abs(float(norm) - n) <= 6 * U * n
    c = min(1.0, max_norm / (n + 1e-6))
    for i, (t, o) in enumerate(zip(ts, outs)):
        want = t.double() * c
        tol = (9 * U + (2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0)) * want.abs()
        assert bool(((o.double() - want).abs() <= tol).all()), (i, t.numel(), t.dtype)


BOTH = (torch.float32, torch.bfloat16)
LISTS = {"one": [1], "some": [5, 0, 64, 100003], "tile edges": [16383, 16384, 16385, 32768, 49151],
         "many small": [1 + 7 * i % 97 for i in range(300)], "exactly two launches": [40] * 256,
         "many tiles": [16384 * 400 + 3, 16384 * 700, 17], "empty": [0, 0]}


@pytest.mark.parametrize("dtypes", [BOTH[:1], BOTH[1:], BOTH], ids=["f32", "bf16", "both"])
@pytest.mark.parametrize("sizes", LISTS.values(), ids=LISTS.keys())
def test_lists(gpu, sizes, dtypes):
    import scan_linear_rnns_amd as mgs
    say(f"clip {len(sizes)} tensors {sum(sizes)} elements")
    ts = tensors(gpu, sizes, dtypes)
    full = math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))
    for max_norm in (full / 3, full * 2, 0.0):
        norm, outs = mgs.mgs_clip_norm(ts, max_norm, out=[torch.empty_like(t) for t in ts])
        check(ts, norm, outs, max_norm)
        if max_norm > full:
            assert all(torch.equal(t, o) for t, o in zip(ts, outs))
    only, none = mgs.mgs_clip_norm(ts)
    assert none is None and torch.equal(only, norm)
    mine = [t.clone() for t in ts]
    norm, same = mgs.mgs_clip_norm(mine, full / 2)
    assert all(a is b for a, b in zip(mine, same))
    check(ts, norm, mine, full / 2)


def test_unaligned_and_shaped(gpu):
    """Views that no wide access may take (odd offsets), among aligned ones; two-dimensional tensors."""
    import scan_linear_rnns_amd as mgs
    say("clip unaligned")
    for dt in BOTH:
        flat = tensors(gpu, [200011], (dt,))[0]
        ts = [flat[1:50000], flat[50001:50003], flat[50008:100008], flat[100008:200008].view(400, 250)]
        out = torch.zeros_like(flat)
        outs = [out[3:50002], out[50004:50006], out[50016:100016], torch.empty(400, 250, dtype=dt, device=gpu)]
        norm, got = mgs.mgs_clip_norm(ts, 1.0, out=outs)
        check(ts, norm, got, 1.0)
        assert out[:3].count_nonzero() == 0 and out[50002:50004].count_nonzero() == 0


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e38])
def test_non_finite_norm_passes_values_through(gpu, value):
    """An infinity, a NaN, and a square past fp32: the norm says so, the values stay."""
    import scan_linear_rnns_amd as mgs
    say(f"clip with {value}")
    ts = tensors(gpu, [1000, 40000])
    ts[1][33333] = value
    norm, outs = mgs.mgs_clip_norm(ts, 1.0, out=[torch.empty_like(t) for t in ts])
    assert not math.isfinite(float(norm))
    assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(ts, outs))


def test_runs_alike_on_any_stream_and_in_graphs(gpu):
    import scan_linear_rnns_amd as mgs
    say("clip determinism, stream, graph")
    ts = tensors(gpu, [100000, 3, 4567] * 50, BOTH)
    outs = [torch.empty_like(t) for t in ts]
    norm, _ = mgs.mgs_clip_norm(ts, 1.0, out=outs)
    first = norm.clone(), [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm, _ = mgs.mgs_clip_norm(ts, 1.0, out=outs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(norm, first[0]) and all(torch.equal(a, b) for a, b in zip(outs, first[1]))
    ws = mgs.workspace(mgs.mgs_clip_norm_workspace_size([t.numel() for t in ts]), gpu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mgs.mgs_clip_norm(ts, 1.0, out=outs, norm=norm, ws=ws)
    for _ in range(3):
        norm.fill_(float("nan"))
        for o in outs:
            o.fill_(float("nan"))
        (torch.randn(1 << 18, device=gpu) * 2).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, first[0]) and all(torch.equal(a, b) for a, b in zip(outs, first[1]))


def test_refusals(gpu):
    import scan_linear_rnns_amd as mgs
    say("clip refusals")
    t = torch.ones(10, 10, device=gpu)
    for bad, err in (([], ValueError), ([t.half()], TypeError), ([t.cpu()], (TypeError, ValueError)),
                     ([t, t.t()[:3]], ValueError), ([t, t.cpu()], (TypeError, ValueError))):
        with pytest.raises(err):
            mgs.mgs_clip_norm(bad, 1.0)
    with pytest.raises(ValueError):
        mgs.mgs_clip_norm([t], 1.0, out=[])
    with pytest.raises(ValueError):
        mgs.mgs_clip_norm([t], 1.0, out=[t[:5]])
    for max_norm in (-1.0, float("nan")):
        with pytest.raises(mgs.MgsError, match="INVALID"):
            mgs.mgs_clip_norm([t], max_norm)
    flat = torch.ones(100, device=gpu)
    with pytest.raises(mgs.MgsError, match="INVALID"):           # shifted over itself
        mgs.mgs_clip_norm([flat[:50]], 1.0, out=[flat[10:60]])
    with pytest.raises(mgs.MgsError, match="WORKSPACE"):
        mgs.mgs_clip_norm([flat], 1.0, ws=torch.empty(16, dtype=torch.uint8, device=gpu))
    assert bool((flat == 1).all()) and bool((t == 1).all())
