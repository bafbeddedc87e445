"""GPU parity of the norm with the residual's addition (mgs_rmsnorm_fwd, _fwd_fp8, _bwd) with its definition in 64
bits.

Tolerances, element by element.  A mean of d squares in fp32 is off by at most (d / 512 + 20) 2^-24 of itself however
its sum is split over lanes (8 neighbours, turns, a tree), and its root by half of that; the products add a few 2^-24:
    y: (d / 512 + 40) 2^-24 |y|;   rstd the same;   h: 2^-24 (|x| + |residual|).
dx subtracts h rstd^3 mean(dy w h) from dy w rstd: the same factor times the absolute values of both.  dw adds `rows`
terms, walked by up to 2048 partial sums: (rows / 512 + 40) 2^-24 times the sum of absolute terms.  An output in bf16
is rounded by at most 2^-8 of itself more.  An 8-bit value is a rounding of y / scale: off by at most 2^-4 of itself,
or half of the smallest step 2^-9 below the smallest normal 2^-6, and by what y and scale are off.
"""
import numpy as np
import pytest
import torch

from tests import layers_reference as ref
from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def within(x, want, tol, who):
    x = n64(x)
    assert x.shape == want.shape, (who, x.shape, want.shape)
    bad = ~(np.abs(x - want) <= tol)
    assert not bad.any(), (who, int(bad.sum()), x[bad][:4], want[bad][:4])


def last_bit(t, want):
    return 2.0 ** -8 * np.abs(want) if t.dtype == torch.bfloat16 else 0.0


def inputs(dev, rows, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = [rand(rows, d), 3 * rand(rows, d), 1 + 0.1 * rand(d), rand(rows, d), rand(rows, d)]
    return [x.to(DT[dtype]).to(dev) for x in t]


def check_fwd(x, res, w, y, h, rstd):
    d = x.shape[-1]
    f = (d / 512 + 40) * 2.0 ** -24
    wy, wh, wr = ref.rmsnorm(n64(x), n64(w), n64(res), EPS)
    within(y, wy, f * np.abs(wy) + last_bit(y, wy), "y")
    within(rstd, wr, f * wr, "rstd")
    size = np.abs(n64(x)) + (0 if res is None else np.abs(n64(res)))
    within(h, wh, 2.0 ** -24 * size + last_bit(h, wh), "h")


def check_bwd(dy, h, w, rstd, dh, dx, dw):
    rows, d = h.reshape(-1, h.shape[-1]).shape
    wx, ww = ref.rmsnorm_bwd(n64(dy), n64(h), n64(w), n64(rstd), n64(dh))
    e, r = np.abs(n64(dy) * n64(w)), n64(rstd)[..., None]
    size = r * (e + np.abs(n64(h)) * r * r * (e * np.abs(n64(h))).mean(-1, keepdims=True))
    size = size + (0 if dh is None else np.abs(n64(dh)))
    within(dx, wx, (d / 512 + 40) * 2.0 ** -24 * size + last_bit(dx, wx), "dx")
    terms = np.abs(n64(dy) * n64(h) * r).reshape(rows, d).sum(0)
    within(dw, ww, (rows / 512 + 40) * 2.0 ** -24 * terms, "dw")


WIDTHS = [1, 7, 8, 64, 100, 511, 512, 513, 1000, 1024, 2048, 2056, 4096, 5000, 8192, 8200, 16384, 20001, 65536]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(gpu, d, dtype):
    import scan_linear_rnns_amd as mgs
    rows = 5 if d > 4096 else 37
    say(f"rmsnorm {rows} x {d} {dtype}")
    x, res, w, dy, dh = inputs(gpu, rows, d, dtype, d)
    y, h, rstd = mgs.mgs_rmsnorm_fwd(x, w, res, eps=EPS)
    check_fwd(x, res, w, y, h, rstd)
    dx, dw = mgs.mgs_rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    check_bwd(dy, h, w, rstd, dh, dx, dw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 64), (3, 100), (2049, 64), (4099, 520), (1500, 2048)])
def test_rows(gpu, rows, d, dtype):
    """Fewer rows than workgroups of the gradient, and more; no residual, no gradient from above."""
    import scan_linear_rnns_amd as mgs
    say(f"rmsnorm {rows} x {d} {dtype} alone")
    x, _, w, dy, _ = inputs(gpu, rows, d, dtype, rows)
    y, h, rstd = mgs.mgs_rmsnorm_fwd(x, w, eps=EPS)
    assert h is x
    check_fwd(x, None, w, y, h, rstd)
    dx, dw = mgs.mgs_rmsnorm_bwd(dy, h, w, rstd)
    check_bwd(dy, h, w, rstd, None, dx, dw)


def test_gradient_against_differences(gpu):
    """A central difference of the 64-bit definition along a random direction; truncation is e^2 = 1e-8 of the third
    derivative (order 10 of the loss's slope here), the kernel's own rounding as above."""
    import scan_linear_rnns_amd as mgs
    say("rmsnorm differences")
    x, _, w, dy, _ = inputs(gpu, 6, 100, "f32", 1)
    _, h, rstd = mgs.mgs_rmsnorm_fwd(x, w, eps=EPS)
    dx, dw = mgs.mgs_rmsnorm_bwd(dy, h, w, rstd)
    r, e = np.random.RandomState(0), 1e-4
    for t, got in ((x, dx), (w, dw)):
        u = r.randn(*t.shape)
        f = lambda s: (ref.rmsnorm(n64(x) + (s * u if t is x else 0), n64(w) + (s * u if t is w else 0), eps=EPS)[0]  # noqa: E731
                       * n64(dy)).sum()
        diff = (f(e) - f(-e)) / (2 * e)
        size = np.abs(n64(got) * u).sum()
        assert abs(diff - (n64(got) * u).sum()) <= 1e-6 * size + 60 * 2.0 ** -24 * size


def check_fp8(x, res, w, y8, scale, h, group):
    d = x.shape[-1]
    wy, wh, _ = ref.rmsnorm(n64(x), n64(w), n64(res), EPS)
    width = group or d
    starts = list(range(0, d, width))
    f = (d / 512 + 44) * 2.0 ** -24
    ws = np.stack([np.maximum(np.abs(wy[:, i:i + width]).max(1), 1e-30) / 448 for i in starts], 1)
    within(scale, ws, f * ws, "scale")
    full = np.repeat(n64(scale), width, axis=1)[:, :d]
    ratio = wy / full
    q = n64(y8.float())
    # what the value is off already may carry it over a rounding boundary, where the error is the larger of both sides'
    within(y8.float(), ratio, 2.0 ** -4 * np.maximum(np.abs(ratio), np.abs(q)) + 2.0 ** -10 + 2 * f * np.abs(ratio), "y8")
    want = torch.from_numpy(ratio).float().to(torch.float8_e4m3fn)
    same = (want.float().numpy() == q).mean()
    assert same >= 0.999, same   # a boundary lies within f of a value about once in 1e5
    size = np.abs(n64(x)) + (0 if res is None else np.abs(n64(res)))
    within(h, wh, 2.0 ** -24 * size + last_bit(h, wh), "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,d", [(1, 128), (9, 64), (33, 127), (65, 129), (7, 1000), (5, 2048), (4, 5000),
                                    (3, 16384), (2, 20001)])
def test_8bit(gpu, rows, d, group, dtype):
    import scan_linear_rnns_amd as mgs
    say(f"rmsnorm fp8 {rows} x {d} group {group} {dtype}")
    x, res, w, _, _ = inputs(gpu, rows, d, dtype, d)
    y8, scale, h = mgs.mgs_rmsnorm_fwd_fp8(x, w, res, eps=EPS, group=group)
    check_fp8(x, res, w, y8, scale, h, group)


def test_8bit_rounds_like_the_type(gpu):
    """Exact midpoints and edges: with rstd one and a scale of one, every rounding is to nearest, ties to even."""
    import scan_linear_rnns_amd as mgs
    say("rmsnorm fp8 ties")
    d = 128
    grid = torch.tensor([448., 1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 17.0, 19.0, 432., 0.0])
    x = torch.ones(1, d, device=gpu)
    w = torch.ones(d)
    w[:grid.numel()] = grid
    y8, scale, _ = mgs.mgs_rmsnorm_fwd_fp8(x, w.to(gpu), eps=0.0)
    assert float(scale) == 1.0
    assert torch.equal(y8[0].float().cpu(), w.to(torch.float8_e4m3fn).float())


def test_rows_of_zeros_and_of_non_finite_values(gpu):
    import scan_linear_rnns_amd as mgs
    say("rmsnorm zeros, NaN, inf")
    x, res, w, dy, dh = inputs(gpu, 8, 300, "f32", 4)
    x[1] = 0
    res[1] = 0
    x[3, 17] = float("nan")
    x[5, 200] = float("inf")
    y, h, rstd = mgs.mgs_rmsnorm_fwd(x, w, res, eps=EPS)
    assert torch.count_nonzero(y[1]) == 0 and torch.isfinite(rstd[1])
    assert torch.isnan(y[3]).all() and torch.isnan(y[5, 200]) and rstd[5] == 0
    for group in (0, 128):
        y8, scale, _ = mgs.mgs_rmsnorm_fwd_fp8(x, w, res, eps=EPS, group=group)
        assert torch.count_nonzero(y8[1].float()) == 0 and bool((scale[1] > 0).all())
        assert torch.isnan(y8[3].float()).all()
        fine = [0, 2, 4, 6, 7]
        check_fp8(x[fine], res[fine], w, y8[fine], scale[fine], h[fine], group)
    dx, _ = mgs.mgs_rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    keep = [0, 1, 2, 4, 6, 7]
    assert torch.isfinite(dx[keep]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_alignment_and_in_place(gpu, dtype):
    import scan_linear_rnns_amd as mgs
    say(f"rmsnorm strides {dtype}")
    x, res, w, dy, dh = inputs(gpu, 40, 256, dtype, 6)
    y0, h0, r0 = mgs.mgs_rmsnorm_fwd(x, w, res, eps=EPS)
    wide = torch.empty(40, 600, dtype=x.dtype, device=gpu)
    for at in (8, 3):                            # a column slice, aligned and not
        wide[:, at:at + 256] = x
        y, h, r = mgs.mgs_rmsnorm_fwd(wide[:, at:at + 256], w, res, eps=EPS)
        assert torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(r, r0)
    flat = torch.empty(256 + 1, dtype=w.dtype, device=gpu)
    flat[1:] = w
    assert torch.equal(mgs.mgs_rmsnorm_fwd(x, flat[1:], res, eps=EPS)[0], y0)
    one = x[:1].expand(40, -1)                   # one row for all
    assert torch.equal(mgs.mgs_rmsnorm_fwd(one, w, eps=EPS)[0], mgs.mgs_rmsnorm_fwd(one.contiguous(), w, eps=EPS)[0])
    stream = res.clone()                         # the residual stream, updated in place
    y, h, _ = mgs.mgs_rmsnorm_fwd(x, w, stream, eps=EPS, h=stream)
    assert h is stream and torch.equal(stream, h0) and torch.equal(y, y0)
    dx0, dw0 = mgs.mgs_rmsnorm_bwd(dy, h0, w, r0, dh=dh)
    for t in (dy.clone(), dh.clone()):
        a, b = (t, dh) if torch.equal(t, dy) else (dy, t)
        dx, dw = mgs.mgs_rmsnorm_bwd(a, h0, w, r0, dh=b, dx=t)
        assert dx is t and torch.equal(dx, dx0) and torch.equal(dw, dw0)
    three = mgs.mgs_rmsnorm_fwd(x.view(4, 10, 256), w, res.view(4, 10, 256), eps=EPS)
    assert three[0].shape == (4, 10, 256) and three[2].shape == (4, 10) and torch.equal(three[0].view(40, 256), y0)


def test_empty_stream_and_refusals(gpu):
    import scan_linear_rnns_amd as mgs
    say("rmsnorm empty, streams, refusals")
    x, res, w, dy, dh = inputs(gpu, 12, 96, "f32", 8)
    y, h, r = mgs.mgs_rmsnorm_fwd(x[:0], w, res[:0])
    dx, dw = mgs.mgs_rmsnorm_bwd(dy[:0], h, w, r)
    assert y.shape == (0, 96) and dx.shape == (0, 96) and torch.count_nonzero(dw) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1 = mgs.mgs_rmsnorm_fwd(x, w, res, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y1, mgs.mgs_rmsnorm_fwd(x, w, res)[0])
    for bad, err in (((x.half(), w), TypeError), ((x.cpu(), w), TypeError), ((x, w[:5]), ValueError),
                     ((x, w.bfloat16()), TypeError), ((x, w, res[:3]), ValueError), ((x.t(), w[:12]), ValueError)):
        with pytest.raises(err):
            mgs.mgs_rmsnorm_fwd(*bad)
    with pytest.raises(mgs.MgsError, match="UNSUPPORTED"):
        mgs.mgs_rmsnorm_fwd_fp8(x, w, group=64)
    with pytest.raises(mgs.MgsError, match="INVALID"):
        mgs.mgs_rmsnorm_fwd(x, w, eps=-1.0)
    with pytest.raises(mgs.MgsError, match="INVALID"):        # h over the weights
        both = torch.zeros(13, 96, device=gpu)
        mgs.mgs_rmsnorm_fwd(x, both[0], h=both[:12])
    with pytest.raises(mgs.MgsError, match="UNSUPPORTED"):
        mgs.mgs_rmsnorm_fwd(torch.zeros(1, 65537, device=gpu), torch.zeros(65537, device=gpu))
    torch.cuda.synchronize()


def test_graph_replays(gpu):
    import scan_linear_rnns_amd as mgs
    say("rmsnorm graph")
    x, res, w, dy, dh = inputs(gpu, 700, 512, "bf16", 10)
    y, h, r = mgs.mgs_rmsnorm_fwd(x, w, res)
    dx, dw = mgs.mgs_rmsnorm_bwd(dy, h, w, r, dh=dh)
    want = [t.clone() for t in (y, h, r, dx, dw)]
    ws = mgs.workspace(mgs.mgs_rmsnorm_workspace_size(700, 512), gpu)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mgs.mgs_rmsnorm_fwd(x, w, res, y=y, h=h, rstd=r)
        mgs.mgs_rmsnorm_bwd(dy, h, w, r, dh=dh, dx=dx, dw=dw, ws=ws)
    for _ in range(3):
        for t in (y, h, r, dx, dw):
            t.fill_(float("nan"))
        (torch.randn(1 << 18, device=gpu) * 2).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, h, r, dx, dw)))
