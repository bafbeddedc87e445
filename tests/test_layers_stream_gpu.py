"""What the layer operators allocate for a call on another stream belongs to
that stream: memory freed to it is handed to its later work alone, never to
work of the current stream that could overtake the call's kernels."""
import pytest
import torch


def calls(mgs, gpu):
    x = torch.randn(64, 4096, device=gpu)
    w = torch.ones(4096, device=gpu)
    q = torch.randn(2, 96, 4, 64, device=gpu)
    g = -torch.rand(2, 96, 4, device=gpu)
    S = torch.zeros(2, 4, 64, 64, device=gpu)
    rstd = torch.ones(64, device=gpu)
    return {
        "fwd": lambda s: mgs.mgs_linattn_fwd(q, q, q, g, stream=s),
        "bwd": lambda s: mgs.mgs_linattn_bwd(q, q, q, g, q, stream=s),
        "step": lambda s: mgs.mgs_linattn_step(q[:, 0], q[:, 0], q[:, 0], g[:, 0], S, stream=s),
        "norm": lambda s: mgs.mgs_rmsnorm_fwd(x, w, x, stream=s),
        "norm8": lambda s: mgs.mgs_rmsnorm_fwd_fp8(x, w, x, stream=s),
        "norm_bwd": lambda s: mgs.mgs_rmsnorm_bwd(x, x, w, rstd, stream=s),
        "clip": lambda s: mgs.mgs_clip_norm([x], out=None, stream=s),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["fwd", "bwd", "step", "norm", "norm8", "norm_bwd", "clip"])
def test_allocations_belong_to_the_stream(gpu, name):
    import scan_linear_rnns_amd as mgs
    call = calls(mgs, gpu)[name]
    here = torch.cuda.current_stream()
    side = torch.cuda.Stream()
    side.wait_stream(here)
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.synchronize()
    got = [t for t in (got if isinstance(got, tuple) else (got,)) if isinstance(t, torch.Tensor)]
    owner = {b["address"]: seg["stream"] for seg in torch.cuda.memory_snapshot() for b in seg["blocks"]}
    fresh = [t for t in got if t.data_ptr() not in inputs_of(call)]
    assert fresh and {owner[t.data_ptr()] for t in fresh} == {side.cuda_stream}


def inputs_of(call):
    return {c.cell_contents.data_ptr() for c in call.__closure__ if isinstance(c.cell_contents, torch.Tensor)}


def test_other_device_is_refused():
    """Kernels run on the current GPU: tensors of another one are refused before any launch."""
    from types import SimpleNamespace
    from scan_linear_rnns_amd import layers
    fake = SimpleNamespace(_C=SimpleNamespace(_cuda_getDevice=lambda: 1, _cuda_getCurrentRawStream=lambda d: 7),
                           cuda=SimpleNamespace(current_device=lambda: 1))
    with pytest.raises(ValueError, match="GPU 0"):
        layers._raw_stream(fake, 0)
    assert layers._raw_stream(fake, 1) == 7
