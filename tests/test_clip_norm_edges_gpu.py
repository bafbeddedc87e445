"""GPU tests of the global gradient norm and clipping (mgs_clip_norm) at edges of its definition.  Tolerances as in
test_clip_norm_gpu.py (its norm's covers sums in fp64, which round once)."""
import math

import pytest
import torch

from tests.test_clip_norm_gpu import BOTH, check, tensors
from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

SIZES = [5, 1000, 16384, 40003, 64]   # tails, whole tiles


@pytest.mark.parametrize("dtypes", [BOTH[:1], BOTH[1:], BOTH], ids=["f32", "bf16", "both"])
@pytest.mark.parametrize("scale", [1e30, 1e20, 3e34, 1e-12, 1e-18, 1e-25, 1e-36])
def test_squares_past_fp32(gpu, scale, dtypes):
    """Elements whose squares overflow fp32, or vanish there: the norm is right, and the values are clipped by it."""
    import scan_linear_rnns_amd as mgs
    say(f"clip elements of {scale}")
    ts = [t * scale for t in tensors(gpu, SIZES, dtypes, 3)]
    max_norm = 1.0 if scale > 1 else 1e-30   # (a norm far under 1e-6 is clipped by max_norm / 1e-6)
    norm, outs = mgs.mgs_clip_norm(ts, max_norm, out=[torch.empty_like(t) for t in ts])
    if scale > 1:
        check(ts, norm, outs, max_norm)
        assert abs(math.sqrt(sum(float((o.double() ** 2).sum()) for o in outs)) - 1.0) < 0.01
    else:
        n = math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))
        assert n > 0 and abs(float(norm) - n) <= 6 * 2.0 ** -24 * n
        same, outs = mgs.mgs_clip_norm(ts, 1.0, out=outs)
        assert torch.equal(same, norm) and all(torch.equal(t, o) for t, o in zip(ts, outs))


def test_one_huge_element_among_small_ones(gpu):
    """An exploding, finite gradient is clipped, wherever it lies: in a wide access, a tail, an unaligned view."""
    import scan_linear_rnns_amd as mgs
    say("clip one huge element")
    for at in (0, 16383, 16384, 40002):
        flat = tensors(gpu, [40004])[0]
        for t in (flat[:40003], flat[1:]):
            t[at] = 7e37
            norm, (out,) = mgs.mgs_clip_norm([t], 1.0, out=[torch.empty_like(t)])
            n = math.sqrt(float((t.double() ** 2).sum()))
            assert abs(float(norm) - n) <= 6 * 2.0 ** -24 * n
            want = t.double() * (1.0 / (n + 1e-6))   # the small ones' are subnormal: half their spacing is 2^-150
            assert bool(((out.double() - want).abs() <= 9 * 2.0 ** -24 * want.abs() + 2.0 ** -150).all()), at
            assert abs(float(out[at]) - 1.0) <= 9 * 2.0 ** -24
            t[at] = 0.0
    ts = tensors(gpu, [1000])
    ts[0][5] = 2.0 ** 126                 # the least norm that counts as not finite
    norm, outs = mgs.mgs_clip_norm(ts, 1.0, out=[torch.empty_like(t) for t in ts])
    assert math.isinf(float(norm)) and torch.equal(ts[0], outs[0])


def test_subnormal_elements(gpu):
    import scan_linear_rnns_amd as mgs
    say("clip subnormal elements")
    t = torch.full((20000,), 1e-40, device=gpu)
    norm, _ = mgs.mgs_clip_norm([t])
    n = math.sqrt(float((t.double() ** 2).sum()))
    assert abs(float(norm) - n) <= 6 * 2.0 ** -24 * n
