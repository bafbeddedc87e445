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
