"""The norm with an eps near the end of fp32's range: mean of squares and eps may each be
finite where their sum is not."""
import numpy as np
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k
from test_gpu_norm import REL, _f64, _formula

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 8, 31, 2056, 4099, 20000])
@pytest.mark.parametrize("eps", [2e36, 1.1e37, 3.4e38])
def test_eps_of_the_largest_numbers(n, eps):
    g = torch.Generator().manual_seed(n)
    base = 1 + torch.rand(1, n, generator=g)
    x = torch.cat([base * s for s in (0.0, 1e-10, 1.0, 1e15, 3e17, 1e18, 1e19, 1e30)])
    y, rstd = torch.empty(x.shape, device="cuda"), torch.empty(x.shape[0], device="cuda")
    k.RmsNorm(n, eps).forward(y, x.cuda(), rstd=rstd)
    want, s = _formula(x.numpy().astype(np.float64), None, np.float64(np.float32(eps)))
    assert (np.abs(_f64(rstd) - s[:, 0]) <= s[:, 0] * REL).all()
    assert (np.abs(_f64(y) - want) <= np.abs(want) * (REL + 2.0 ** -24) + 1e-38).all()
