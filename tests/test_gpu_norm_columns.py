"""The gradient of the norm's gains where the order of its additions shows: one large term
and ones that are half of its last place, which a sum of one after the other loses."""
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# n, rows, rows of a CTA at a time (those between are zeros): a part of the column sums for
# each of 32 warps
@pytest.mark.parametrize("dt,n,T,step", [("f32", 1024, 64, 2), ("f32", 9000, 32, 1), ("bf16", 2000, 64, 2),
                                         ("bf16", 9000, 32, 1)])
def test_small_terms_beside_a_large_one(dt, n, T, step):
    r = torch.ones(T, n, dtype=DT[dt], device="cuda")
    dy = torch.zeros(T, n, dtype=DT[dt], device="cuda")
    dy[::step] = 1
    dy[0] = 2.0 ** 24  # the next fp32 number is 2 further
    gain, rstd = torch.ones(n, device="cuda"), torch.ones(T, device="cuda")
    dx, dgain = torch.empty_like(r), torch.empty(n, device="cuda")
    norm = k.RmsNorm(n, 1e-6)
    norm.backward(dx, dgain, dy, r, rstd, gain)
    want = 2.0 ** 24 + T // step - 1
    # the large term is part of eight additions at most: a row's, two of a CTA's teams, a
    # warp's parts, five that join 32 warps; each loses half a step of 2 at most.  (One warp
    # after the other 31 of them do.)
    assert float((dgain.double() - want).abs().max()) <= 9
    norm.backward(dx, dgain, dy, r, rstd, gain, accumulate=True)
    assert float((dgain.double() - 2 * want).abs().max()) <= 2 * 9 + 2
