"""Quantisation of rows near the longest that an operand may have (2^30 columns):
codes and scale atoms equal those of the row's pieces quantised one by one."""
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
PIECE = 1 << 26


def _room(n):
    if torch.cuda.mem_get_info()[0] < n:
        pytest.skip("needs %.0f GB of device memory" % (n / 1e9))


@pytest.mark.parametrize("cols,dt", [((1 << 29) - 128, torch.float32), (1 << 29, torch.float32),
                                     ((1 << 29) + 52, torch.float32), (1 << 30, torch.float32),
                                     (1 << 30, torch.bfloat16)])
def test_one_long_row(cols, dt):
    _room(24 << 30)
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(1, cols, generator=g, device="cuda", dtype=dt)
    op = k.MxOperand(1, cols)
    k.mx_quantize_operand(x, op)
    for a in range(0, cols, PIECE):
        n = min(PIECE, cols - a)
        part = k.MxOperand(1, n)
        k.mx_quantize_operand(x[:, a:a + n], part)
        assert torch.equal(op.codes[a // 2:a // 2 + part.codes.numel()], part.codes), a
        at = a // 128 * 512
        assert torch.equal(op.atoms[at:at + part.atoms.numel()], part.atoms), a
        assert bool(part.codes.any())
    assert k.device_error() == 0


def test_one_long_row_by_its_columns():
    """The same along the other axis: 2^29 rows of one value each."""
    _room(40 << 30)
    cols = (1 << 29) + 52
    x = torch.randn(1, cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    op = k.MxOperand(cols, 1)
    k.mx_quantize_operand(x, None, op)
    for a in range(0, cols, PIECE):
        n = min(PIECE, cols - a)
        part = k.MxOperand(n, 1)
        k.mx_quantize_operand(x[:, a:a + n], None, part)
        assert torch.equal(op.codes[a * 16:(a + n) * 16], part.codes), a
        at = a // 128 * 1024
        assert torch.equal(op.atoms[at:at + part.atoms.numel()], part.atoms), a
        assert bool(part.codes.any())
    assert k.device_error() == 0
