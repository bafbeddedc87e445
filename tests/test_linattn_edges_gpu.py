"""GPU tests of linear attention (mgs_linattn_fwd, _bwd, _step) at edges of its definition: empty batches, cleared
states, variants that only some calls reach.  Tolerances as in test_linattn_gpu.py where nothing else is said."""
import pytest
import torch

from tests.test_linattn_gpu import make, run
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
