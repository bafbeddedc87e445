"""GPU tests of the norm with the residual's addition (mgs_rmsnorm_fwd, _fwd_fp8, _bwd) at edges of its definition."""
import pytest
import torch

from tests.test_parity_gpu import say
from tests.test_rmsnorm_gpu import EPS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,d", [(4096, 1000), (2000, 2048), (3000, 999), (600, 8200)])
def test_8bit_is_the_rounded_quotient(gpu, rows, d, group):
    """y8 is y / scale rounded, bit for bit, for the fp32 y and scale that the same inputs give: bf16 inputs and weights
    make quotients that lie on ties.  (The division and the rounding are taken on the CPU.)"""
    import scan_linear_rnns_amd as mgs
    say(f"rmsnorm fp8 quotients {rows} x {d} group {group}")
    gen = torch.Generator().manual_seed(d + group)
    x = torch.randn(rows, d, generator=gen).bfloat16().to(gpu)
    w = (1 + 0.1 * torch.randn(d, generator=gen)).bfloat16().to(gpu)
    y8, scale, _ = mgs.mgs_rmsnorm_fwd_fp8(x, w, eps=EPS, group=group)
    y = mgs.mgs_rmsnorm_fwd(x.float(), w.float(), eps=EPS)[0].cpu()
    width = group or d
    y = torch.nn.functional.pad(y, (0, -d % width)).unflatten(1, (-1, width))
    want = y.abs().amax(-1) / 448.0
    assert torch.equal(scale.cpu(), want)
    q = (y / want[..., None]).flatten(1)[:, :d].to(torch.float8_e4m3fn)
    assert torch.equal(y8.cpu().view(torch.uint8), q.view(torch.uint8))
