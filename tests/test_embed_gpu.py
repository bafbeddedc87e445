"""GPU parity of the embedding lookup and its gradient (mgs_embed_fwd, mgs_embed_bwd) with their definitions in 64
bits.

Tolerances, element by element: y is one product, rounded to fp32 and to the output's type: 2^-24 |y| and, in bf16,
2^-8 |y| more.  dW of m rows is added up in chunks of 32 and these among four shares: at most 32 + m / 32 + 4 additions
one after another and one product, each off by 2^-24 of the sum of absolute values; an addition to what dW held before
is one more of |before| too."""
import numpy as np
import pytest
import torch

from tests import tokens_reference as ref
from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def n64(t):
    return t.detach().double().cpu().numpy()


def within(x, want, tol, who):
    x = n64(x).reshape(want.shape)
    bad = ~(np.abs(x - want) <= tol)
    assert not bad.any(), (who, int(bad.sum()), x[bad][:4], want[bad][:4])


def last_bit(t, want):
    return 2.0 ** -8 * np.abs(want) if t.dtype == torch.bfloat16 else 0.0


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def check_bwd(ids, dy, vocab, scale, dW, before=None):
    want, size, many = ref.embed_bwd(ids.cpu().numpy(), n64(dy), vocab, scale)
    if before is not None:
        want, size = want + n64(before), size + np.abs(n64(before))
    within(dW, want, (38 + many[:, None] / 32) * 2.0 ** -24 * size + last_bit(dW, want), "dW")


def random_ids(n, vocab, seed, outside=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (n,), generator=g)
    bad = torch.tensor([-1, vocab, -2 ** 40, 2 ** 40])[torch.randint(0, 4, (n,), generator=g)]
    return ids.where(torch.rand(n, generator=g) > outside, bad)


SIZES = [(1, 1, 1), (1, 5, 8), (3, 2, 7), (33, 64, 9), (64, 65, 64), (100, 3, 100), (257, 1000, 24), (1000, 129, 513),
         (31, 70000, 40), (2000, 300, 2056), (5, 9, 20000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,d", SIZES)
def test_sizes(gpu, n, vocab, d, dtype):
    import scan_linear_rnns_amd as mgs
    say(f"embed n={n} vocab={vocab} d={d} {dtype}")
    ids = random_ids(n, vocab, n + vocab).to(gpu)
    W, dy = randn(vocab, d, seed=1).to(DT[dtype]).to(gpu), randn(n, d, seed=2).to(DT[dtype]).to(gpu)
    y = mgs.mgs_embed_fwd(ids, W, scale=1.7)
    want = ref.embed(ids.cpu().numpy(), n64(W), float(np.float32(1.7)))
    within(y, want, 2.0 ** -24 * np.abs(want) + last_bit(y, want), "y")
    for out in (torch.float32, torch.bfloat16):
        check_bwd(ids, dy, vocab, float(np.float32(0.3)), mgs.mgs_embed_bwd(ids, dy, vocab, scale=0.3, dtype=out))


@pytest.mark.parametrize("n,vocab,many", [(5000, 50, 1), (4096, 700, 3), (70000, 5, 2), (3000, 40000, 1)])
def test_few_ids_are_most_of_the_text(gpu, n, vocab, many):
    """Runs of one id over many chunks, starting and ending at and off their borders."""
    import scan_linear_rnns_amd as mgs
    say(f"embed heavy ids n={n} vocab={vocab}")
    ids = random_ids(n, vocab, n, 0.01)
    g = torch.Generator().manual_seed(n)
    for i in range(many):
        ids = ids.where(torch.rand(n, generator=g) > 0.6, (i * 31) % vocab)
    ids, dy = ids.to(gpu), randn(n, 72, seed=3).to(gpu)
    check_bwd(ids, dy, vocab, 1.0, mgs.mgs_embed_bwd(ids, dy, vocab))


@pytest.mark.parametrize("n", [32, 64, 96, 97, 4096])
@pytest.mark.parametrize("vocab", [1, 130])
def test_one_id(gpu, n, vocab):
    import scan_linear_rnns_amd as mgs
    say(f"embed one id n={n} vocab={vocab}")
    ids, dy = torch.full((n,), vocab - 1, device=gpu), randn(n, 16, seed=4).to(gpu)
    check_bwd(ids, dy, vocab, 1.0, mgs.mgs_embed_bwd(ids, dy, vocab))


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_accumulate(gpu, dtype, out):
    """Added to what dW holds; rows of ids that do not occur are left alone, NaN and all."""
    import scan_linear_rnns_amd as mgs
    say(f"embed accumulate {dtype} {out}")
    n, vocab, d = 500, 90, 40
    m = vocab // 2
    ids = random_ids(n, m, 5)
    ids = ids.where((ids >= 0) & (ids < m), -1).to(torch.int32).to(gpu)   # (m itself is a row of this table)
    dy, dW = randn(n, d, seed=6).to(DT[dtype]).to(gpu), randn(vocab, d, seed=7).to(DT[out]).to(gpu)
    dW[m + 3:] = float("nan")
    before = dW.clone()
    got = mgs.mgs_embed_bwd(ids, dy, vocab, scale=2.0, dW=dW, accumulate=True)
    assert got is dW and torch.equal(dW[m:].view(torch.uint8), before[m:].view(torch.uint8))
    check_bwd(ids, dy, m, 2.0, dW[:m], before[:m])


def test_strides_alignment_and_shapes(gpu):
    """Rows apart, rows that no wide access can take, ids of several dimensions: the same bits."""
    import scan_linear_rnns_amd as mgs
    say("embed strides")
    vocab, d = 77, 64
    for dt in (torch.float32, torch.bfloat16):
        wide = randn(vocab, 100, seed=8).to(dt).to(gpu)
        ids = random_ids(60, vocab, 9).view(4, 15).to(gpu)
        dy = randn(60, 130, seed=10).to(dt).to(gpu)
        for off in (0, 3, 8):
            W, g = wide[:, off:off + d], dy[:, off:off + d]
            y = mgs.mgs_embed_fwd(ids, W)
            assert y.shape == (4, 15, d) and torch.equal(y, mgs.mgs_embed_fwd(ids, W.contiguous()))
            dW = mgs.mgs_embed_bwd(ids.view(60), g, vocab)
            assert torch.equal(dW, mgs.mgs_embed_bwd(ids, g.contiguous().view(4, 15, d), vocab))
        raw = torch.empty(vocab * d + 3, dtype=dt, device=gpu)
        odd = mgs.mgs_embed_bwd(ids.view(60), g, vocab, dW=raw[3:].view(vocab, d), dtype=dt)
        assert torch.equal(odd, mgs.mgs_embed_bwd(ids.view(60), g, vocab, dtype=dt))
        # one row for all places
        same = dy[:1, :d].expand(60, d)
        assert torch.equal(mgs.mgs_embed_bwd(ids.view(60), same, vocab),
                           mgs.mgs_embed_bwd(ids.view(60), same.contiguous(), vocab))


def test_empty(gpu):
    import scan_linear_rnns_amd as mgs
    say("embed empty")
    W = randn(5, 8, seed=1).to(gpu)
    none = torch.empty(0, dtype=torch.int64, device=gpu)
    assert mgs.mgs_embed_fwd(none, W).shape == (0, 8)
    assert mgs.mgs_embed_fwd(torch.tensor([0, 3], device=gpu), W[:0]).count_nonzero() == 0
    dW = mgs.mgs_embed_bwd(none, W[:0], 5, dW=torch.full((5, 8), float("nan"), device=gpu))
    assert torch.equal(dW, torch.zeros(5, 8, device=gpu))
    assert mgs.mgs_embed_bwd(none, W[:0], 5, dW=W.clone(), accumulate=True).equal(W)
    assert mgs.mgs_embed_bwd(none, W[:0], 0).shape == (0, 8)
    pad = torch.full((40,), -1, device=gpu)
    assert mgs.mgs_embed_bwd(pad, randn(40, 8, seed=2).to(gpu), 5).count_nonzero() == 0


def test_same_bits_every_time(gpu):
    import scan_linear_rnns_amd as mgs
    say("embed determinism")
    ids = (torch.rand(20000, generator=torch.Generator().manual_seed(1)) ** 4 * 3000).long().to(gpu)
    dy = randn(20000, 136, seed=2).to(gpu)
    one = mgs.mgs_embed_bwd(ids, dy, 3000)
    ws = torch.randint(0, 255, (mgs.mgs_embed_workspace_size(20000, 3000, 136),), dtype=torch.uint8, device=gpu)
    for _ in range(5):
        assert torch.equal(mgs.mgs_embed_bwd(ids, dy, 3000, ws=ws), one)
