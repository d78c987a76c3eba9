"""Outputs on top of inputs: the SwiGLU gradients may take the place of dh row by
row, so only with its stride (no GPU: refused before any CUDA call)."""
import pytest

from mxfp4_routed_expert_select_gb300 import k3moe as k

P, Q = 4096, 1 << 20  # pointers that are never followed


@pytest.mark.parametrize("dg,lddg,du,lddu,dh,lddh", [(P, 80, Q, 40, P, 40), (P, 40, Q, 40, P, 80), (Q, 40, P, 48, P, 40),
                                                     (Q, 40, P, 40, P, 48)])
def test_swiglu_backward_on_dh_with_another_stride(dg, lddg, du, lddu, dh, lddh):
    L = k.lib()
    T, f = 4, 40
    n = L.k3moe_swiglu_ckpt_bytes(T, f)
    for dt in (k.K3MOE_F32, k.K3MOE_BF16):
        assert L.k3moe_swiglu_backward(dg, lddg, du, lddu, dh, lddh, P, n, dt, T, f, None) == k.K3MOE_EINVAL
