"""The query of a product's form: refusals and plain facts (no GPU needed)."""
import ctypes

import pytest

from mxfp4_routed_expert_select_gb300 import k3moe as k


def test_refusals():
    L = k.lib()
    o = [ctypes.byref(ctypes.c_int32()) for _ in range(3)]
    assert L.k3moe_mx_matmul_form(1, 1, 1, k.K3MOE_F32, *o) == k.K3MOE_OK
    big = (1 << 30) + 1
    for M, N, n, dt in ((0, 1, 1, 0), (1, 0, 1, 0), (1, 1, 0, 0), (big, 1, 1, 0), (1, big, 1, 0), (1, 1, big, 0), (1, 1, 1, 2)):
        assert L.k3moe_mx_matmul_form(M, N, n, dt, *o) == k.K3MOE_EINVAL
    for i in range(3):
        p = list(o)
        p[i] = None
        assert L.k3moe_mx_matmul_form(1, 1, 1, k.K3MOE_F32, *p) == k.K3MOE_EINVAL


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 7168, 1536), (33, 1000, 7000), (5000, 5000, 5000), (1 << 20, 64, 32)])
def test_a_form_that_exists(M, N, K):
    torch = pytest.importorskip("torch")
    for dt in (torch.float32, torch.bfloat16):
        pair, columns, ranks = k.mx_matmul_form(M, N, K, dt)
        assert columns in ((192, 256, 384) if pair else (16, 32, 64, 128)) and ranks in ((1,) if pair else (1, 2, 4, 8))
