"""What the token path's operators write into a workspace."""
import pytest
import torch

from tests.test_parity_gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_recurrences_header_is_left_alone(gpu, dtype):
    """The first 256 bytes hold the recurrence's launch words and how long it waits: sampling, in as many slices as there
    are, and the table's gradient leave them as they are, so that no wait is without end on a workspace in common."""
    import scan_linear_rnns_amd as mgs
    say(f"tokens header {dtype}")
    g = torch.Generator().manual_seed(1)
    ws = mgs.workspace(max(mgs.mgs_sample_workspace_size(1, 1 << 20, dtype), mgs.mgs_sample_workspace_size(128, 70000, dtype),
                           mgs.mgs_embed_workspace_size(9000, 5000, 64)), gpu)
    ws.fill_(0xA5)
    before = ws[:256].clone()
    for B, V in ((1, 1 << 20), (128, 70000)):
        x, u = torch.randn(B, V, generator=g).to(dtype).to(gpu), torch.rand(B, generator=g).to(gpu)
        for s in (dict(), dict(top_k=50, top_p=0.9), dict(top_p=0.9), dict(min_p=0.1), dict(temperature=0.0)):
            own = mgs.mgs_sample(x, u, **s)
            for a, b in zip(mgs.mgs_sample(x, u, **s, ws=ws), own):
                assert torch.equal(a, b), (B, V, s)
            assert torch.equal(ws[:256], before), (B, V, s)
    ids, dy = torch.randint(-1, 5000, (9000,), generator=g).to(gpu), torch.randn(9000, 64, generator=g).to(dtype).to(gpu)
    own = mgs.mgs_embed_bwd(ids, dy, 5000)
    assert torch.equal(mgs.mgs_embed_bwd(ids, dy, 5000, ws=ws), own) and torch.equal(ws[:256], before)
