"""The binding of the operand, SwiGLU and balance calls refuses tensors that are not
on their objects' GPU before the library sees a pointer; masks of bytes or bools."""
import pytest

from mxfp4_routed_expert_select_gb300 import k3moe as k

torch = pytest.importorskip("torch")


@pytest.fixture(params=["objects on the CPU too", "objects on GPU 0"])
def on(request):
    """Sets the GPU that an object says it is on."""
    def set_gpu(o):
        if request.param.endswith("0"):
            o.gpu = 0
        return o
    return set_gpu


def _op(on, rows, n):
    return on(k.MxOperand(rows, n, device="cpu"))


def test_operands(on):
    x, A, B, C = torch.zeros(4, 64), _op(on, 4, 64), _op(on, 64, 4), _op(on, 8, 64)
    for row, col in ((A, None), (None, B), (A, B)):
        with pytest.raises(ValueError, match="GPU"):
            k.mx_quantize_operand(x, row, col)
    with pytest.raises(ValueError, match="GPU"):
        k.mx_dequantize(x, A)
    with pytest.raises(ValueError, match="GPU"):
        k.mx_matmul(torch.zeros(4, 8), A, C)
    with pytest.raises(ValueError, match="GPU"):
        k.MxOperand.from_matrix(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), 4, 64)


def test_swiglu(on):
    g, ck = torch.zeros(4, 40), on(k.SwigluCheckpoint(4, 40, device="cpu"))
    with pytest.raises(ValueError, match="GPU"):
        k.swiglu_forward(g, ck, g, g)
    with pytest.raises(ValueError, match="GPU"):
        k.swiglu_backward(g, g.clone(), g, ck)


def test_balance(on):
    bal = on(k.BalanceLoss(8, 2, 0.1, device="cpu"))
    f, i = torch.zeros(1), torch.zeros(1, dtype=torch.int32)
    l, ids, counts = torch.zeros(5, 8), torch.zeros(5, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        bal.forward(f, counts, i, l, ids)
    with pytest.raises(ValueError, match="GPU"):
        bal.backward(torch.empty_like(l), l, ids, counts, i, f)


def test_masks_of_bytes_and_bools():
    bal = k.BalanceLoss(8, 2, 0.1, device="cpu")
    for dt in (torch.uint8, torch.bool):
        m = torch.ones(5, dtype=dt)
        assert bal._mask(m, 5) == m.data_ptr()
    assert bal._mask(None, 5) is None
    for bad in (torch.ones(5), torch.ones(5, dtype=torch.int8), torch.ones(4, dtype=torch.bool),
                torch.ones(10, dtype=torch.bool)[::2]):
        with pytest.raises(ValueError):
            bal._mask(bad, 5)
