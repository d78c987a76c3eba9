"""The combine's weight gradients with rows of several steps of a CTA, at each number of
threads that a CTA has (512, 256 and 128 by the number of CTAs)."""
import numpy as np
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k
from test_gpu_groups import DT, HALF, _case, _gathered

pytestmark = pytest.mark.gpu


# CTAs are ceil(top_k / 4) a token: 40, 400 and 600 of them on 152 SMs
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [4104, 4100])  # rows of whole 16-byte units and not
@pytest.mark.parametrize("T,kk,threads", [(40, 4, 512), (200, 8, 256), (600, 4, 128)])
def test_weight_gradients_of_long_rows(T, kk, threads, n, dt):
    g, ids, y, dout, w = _case(T, kk, 11, n, dt, T + n)
    dy, dw = torch.zeros_like(y), torch.full((T, kk), 9.0, device="cuda")
    k.combine_backward(dy, dw, dout, y, g, w)
    Y, pos = _gathered(ids, 11, y)
    W, D = w.double().cpu().numpy(), dout.double().cpu().numpy()
    want = np.zeros((T * kk, n))
    t, j = np.nonzero(pos >= 0)
    want[pos[t, j]] = W[t, j][:, None] * D[t]
    assert (np.abs(dy.double().cpu().numpy() - want) <= np.abs(want) * HALF[dt]).all()
    # a thread's products one after the other, eight a step; five steps join a warp, then
    # one for each warp
    terms = 8 * -(-n // (8 * threads)) + 5 + threads // 32
    want, mag = np.einsum("tkn,tn->tk", Y, D), np.einsum("tkn,tn->tk", np.abs(Y), np.abs(D))
    assert (np.abs(dw.double().cpu().numpy() - want) <= mag * terms * 2.0 ** -24).all()
    assert bool((dw[torch.from_numpy(pos < 0).cuda()] == 0).all())
