"""Layer operators on grids past one launch (2^32 threads along a dimension): every output is written, and sequences or
rows at the ends, at the launches' seam and anywhere equal, bit for bit, the same call on those alone."""
import gc

import pytest
import torch

from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def freed(gpu):
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def picks(n, seam, dev):
    """Indexes near both ends and the seam, and a few between."""
    at = [0, 1, seam - 1, seam, seam + 1, n - 2, n - 1] + [n * i // 11 for i in range(1, 11)]
    return torch.tensor(sorted({i for i in at if 0 <= i < n}), device=dev)


def randn(*shape, dev, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator(dev).manual_seed(seed), device=dev, dtype=dtype)


def test_norm_rows(gpu):
    """Four rows to a workgroup of 256 threads: 2^26 rows are one launch's limit."""
    import scan_linear_rnns_amd as mgs
    rows, d = (1 << 26) + 5, 8
    say(f"rmsnorm {rows} x {d}")
    x, w = randn(rows, d, dev=gpu, dtype=torch.bfloat16), randn(d, dev=gpu, dtype=torch.bfloat16, seed=1)
    y, rstd = torch.full_like(x, float("nan")), torch.full((rows,), float("nan"), device=gpu)
    mgs.mgs_rmsnorm_fwd(x, w, y=y, rstd=rstd)
    assert bool(torch.isfinite(rstd).all()) and bool(torch.isfinite(y).all())
    at = picks(rows, (1 << 26) - 32, gpu)
    one = mgs.mgs_rmsnorm_fwd(x[at], w)
    assert torch.equal(y[at], one[0]) and torch.equal(rstd[at], one[2])
    scale = torch.full((rows, 1), float("nan"), device=gpu)
    y8, _, _ = mgs.mgs_rmsnorm_fwd_fp8(x, w, scale=scale)
    one = mgs.mgs_rmsnorm_fwd_fp8(x[at], w)
    assert bool(torch.isfinite(scale).all())
    assert torch.equal(y8[at].view(torch.uint8), one[0].view(torch.uint8)) and torch.equal(scale[at], one[1])


def test_attention_sequences(gpu):
    """Sequences of one step, a workgroup of 256 threads for each and role: 2^24 are a forward launch's limit, half of
    that the gradient's."""
    import scan_linear_rnns_amd as mgs
    B, d = (1 << 24) + 9, 8
    say(f"linattn B={B} T=1 d={d}")
    q, k, v, do = (randn(B, 1, 1, d, dev=gpu, seed=i) for i in range(4))
    g = -randn(B, 1, 1, dev=gpu, seed=4).abs()
    S0 = randn(B, 1, d, d, dev=gpu, seed=5)
    at = torch.cat([picks(B, (1 << 24) - 8, gpu), picks(B, (1 << 23) - 4, gpu)]).unique()
    part = [t[at] for t in (q, k, v, g)]
    o, ST = torch.full_like(v, float("nan")), torch.full_like(S0, float("nan"))
    mgs.mgs_linattn_fwd(q, k, v, g, S0=S0, o=o, ST=ST)
    one = mgs.mgs_linattn_fwd(*part, S0=S0[at])
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(ST).all())
    assert torch.equal(o[at], one[0]) and torch.equal(ST[at], one[1])
    outs = (torch.full_like(q, float("nan")), torch.full_like(k, float("nan")), torch.full_like(v, float("nan")),
            torch.full_like(g, float("nan")), torch.full_like(S0, float("nan")))
    mgs.mgs_linattn_bwd(q, k, v, g, do, S0=S0, out=outs)
    # (as many that the same kernels take them: over 256)
    pad = torch.arange(300, device=gpu)
    both = torch.cat([at, pad])
    one = mgs.mgs_linattn_bwd(*(t[both] for t in (q, k, v, g, do)), S0=S0[both])
    for name, t, u in zip(("dq", "dk", "dv", "dg", "dS0"), outs, one):
        assert bool(torch.isfinite(t).all()), name
        assert torch.equal(t[both], u), name


def test_attention_steps(gpu):
    import scan_linear_rnns_amd as mgs
    B, d = (1 << 24) + 9, 8
    say(f"linattn step B={B} d={d}")
    q, k, v = (randn(B, 1, d, dev=gpu, seed=i) for i in range(3))
    g = -randn(B, 1, dev=gpu, seed=4).abs()
    S = randn(B, 1, d, d, dev=gpu, seed=5)
    at = picks(B, (1 << 24) - 8, gpu)
    mine = S[at]
    o = torch.full_like(v, float("nan"))
    mgs.mgs_linattn_step(q, k, v, g, S, o=o)
    one = mgs.mgs_linattn_step(q[at], k[at], v[at], g[at], mine)
    assert bool(torch.isfinite(o).all()) and torch.equal(o[at], one) and torch.equal(S[at], mine)


def test_attention_shared_heads(gpu):
    """dq and dk of 2^32 elements, summed over two heads each."""
    import scan_linear_rnns_amd as mgs
    B, T, H, dk, dv = (1 << 16) + 3, 512, 2, 128, 8
    say(f"linattn B={B} T={T} H={H} on 1, dk={dk}: dq of {B * T * dk} elements")
    q, k = (randn(B, T, 1, dk, dev=gpu, dtype=torch.bfloat16, seed=i) for i in range(2))
    v, do = (randn(B, T, H, dv, dev=gpu, dtype=torch.bfloat16, seed=i) for i in (2, 3))
    g = -randn(B, T, H, dev=gpu, seed=4).abs()
    dq, dkk, dvv = torch.full_like(q, float("nan")), torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    dg = torch.full_like(g, float("nan"))
    mgs.mgs_linattn_bwd(q, k, v, g, do, scale=0.1, out=(dq, dkk, dvv, dg, None))
    # (as many that none is cut into segments, as none is above: over 512 / 6)
    at = torch.cat([picks(B, (1 << 16) - 1, gpu), torch.arange(300, device=gpu)])
    part = [t[at] for t in (q, k, v, g, do)]
    one = [torch.empty_like(t) for t in (part[0], part[1], part[2], part[3])]
    mgs.mgs_linattn_bwd(*part, scale=0.1, out=(*one, None))
    for name, t, u in zip(("dq", "dk", "dv", "dg"), (dq, dkk, dvv, dg), one):
        for i in range(0, B, 4096):
            assert bool(torch.isfinite(t[i:i + 4096]).all()), (name, i)
        assert torch.equal(t[at], u), name


def test_states_of_empty_sequences(gpu):
    """T = 0: 2^32 state elements are copied."""
    import scan_linear_rnns_amd as mgs
    B, d = (1 << 18) + 1, 128
    say(f"linattn T=0, {B * d * d} state elements")
    q, v, g = torch.empty(B, 0, 1, d, device=gpu), torch.empty(B, 0, 1, d, device=gpu), torch.empty(B, 0, 1, device=gpu)
    S0 = randn(B, 1, d, d, dev=gpu)
    ST = torch.full_like(S0, float("nan"))
    mgs.mgs_linattn_fwd(q, q, v, g, S0=S0, ST=ST)
    for i in range(0, B, 16384):
        assert torch.equal(ST[i:i + 16384], S0[i:i + 16384]), i
