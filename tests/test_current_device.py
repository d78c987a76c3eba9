"""The calls of the binding that know their GPU are refused while another device is the
current one: their kernels would run there, on pointers of this one.  (No GPU: objects and
tensors on the CPU, which calls itself device -1.)"""
import pytest

from mxfp4_routed_expert_select_gb300 import k3moe as k

torch = pytest.importorskip("torch")


class Library:
    """Every entry point: counts the calls, all succeed."""
    calls = 0

    def __getattr__(self, name):
        def entry(*args):
            self.calls += 1
            return 0
        return entry


def _calls():
    """Every such call, with tensors that it takes."""
    f, i, b = torch.zeros, torch.int32, torch.bfloat16
    op, ck, bal = k.MxOperand(4, 64, device="cpu"), k.SwigluCheckpoint(4, 64, device="cpu"), k.BalanceLoss(8, 2, 0.1, device="cpu")
    rows, norm, g = k.Mx8Rows(4, 128, device="cpu"), k.RmsNorm(128, 1e-6, device="cpu"), k.ExpertGroups(3, 2, 4, device="cpu")
    W = k.MxExperts(3, 40, 128, device="cpu")
    g.tokens, g.slots, g.struct.tokens = 4, 8, 4
    x, u8 = f(4, 64), lambda *s: f(*s, dtype=torch.uint8)
    n = lambda: f(4, 128)  # noqa: E731
    return dict(
        mx_quantize_operand=lambda: k.mx_quantize_operand(x, op), mx_dequantize=lambda: k.mx_dequantize(x, op),
        mx_from_matrix=lambda: k.MxOperand.from_matrix(u8(4, 32), u8(4, 2), 4, 64),
        mx_matmul=lambda: k.mx_matmul(f(4, 4), op, op), swiglu_forward=lambda: k.swiglu_forward(f(4, 64), ck, x, x),
        swiglu_backward=lambda: k.swiglu_backward(f(4, 64), f(4, 64), x, ck), mx8_quantize=lambda: k.mx8_quantize(rows, n()),
        mx8_dequantize=lambda: k.mx8_dequantize(n(), rows), norm_forward=lambda: norm.forward(n(), n(), y8=rows),
        norm_backward=lambda: norm.backward(n(), None, n(), n(), f(4)), plan=lambda: g.plan(f(4, 2, dtype=i)),
        experts=lambda: k.MxExperts.from_matrices(u8(3, 40, 64), u8(3, 40, 4)),
        grouped_matmul=lambda: k.grouped_matmul(f(8, 40), rows, W, g, gather=True),
        grouped_wgrad=lambda: k.grouped_wgrad(f(3, 40, 128), f(8, 40, dtype=b), f(4, 128, dtype=b), g, gather=True),
        combine=lambda: k.combine(n(), f(8, 128), g), combine_backward=lambda: k.combine_backward(f(8, 128), None, n(), None, g),
        balance_forward=lambda: bal.forward(f(1), f(8, dtype=i), f(1, dtype=i), f(5, 8), f(5, 2, dtype=i)),
        balance_backward=lambda: bal.backward(f(5, 8), f(5, 8), f(5, 2, dtype=i), f(8, dtype=i), f(1, dtype=i), f(1)))


NAMES = list(_calls())


@pytest.fixture
def calls(monkeypatch):
    monkeypatch.setattr(k, "_gpu", lambda t: t.get_device())
    made = _calls()
    real = k.lib()
    lib = Library()
    # sizes of objects made in the calls
    for name in ("k3moe_mx_operand_codes_bytes", "k3moe_mx_operand_atoms_bytes"):
        setattr(lib, name, getattr(real, name))
    monkeypatch.setattr(k, "_lib", lib)
    monkeypatch.setattr(k, "_raw_stream", lambda device: 0)
    return made, lib


@pytest.mark.parametrize("name", NAMES)
def test_another_current_device(monkeypatch, calls, name):
    made, lib = calls
    monkeypatch.setattr(k, "_raw_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        made[name]()
    assert lib.calls == 0
    monkeypatch.setattr(k, "_raw_device", lambda: -1)
    made[name]()
    assert lib.calls == 1


def test_a_stream_does_not_stand_for_its_device(monkeypatch, calls):
    monkeypatch.setattr(k, "_raw_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        k._stream_on(0, 64)
    assert k._stream_on(1, 64) == 64 and k._stream_on(1) == 0
