"""A plan that was not made leaves the object with the plan it had: the grouped calls check
their tensors by its slots and the kernels read by its tokens."""
import ctypes

import pytest

from mxfp4_routed_expert_select_gb300 import k3moe as k

torch = pytest.importorskip("torch")


class Library:
    """The plan's entry point: takes a plan, refuses it, or raises."""

    def __init__(self, result):
        self.result = result

    def k3moe_groups_plan(self, ref, ids, stream):
        if isinstance(self.result, BaseException):
            raise self.result
        return self.result

    def k3moe_strerror(self, st):
        return b"refused"


@pytest.mark.parametrize("result", [k.K3MOE_EINVAL, ctypes.ArgumentError("stream"), KeyboardInterrupt()])
def test_a_plan_that_was_not_made(monkeypatch, result):
    g = k.ExpertGroups(3, 2, 8, device="cpu")
    g.gpu = -1  # as the CPU's tensors say
    monkeypatch.setattr(k, "_raw_device", lambda: -1)
    monkeypatch.setattr(k, "_lib", Library(0))
    g.plan(torch.zeros(3, 2, dtype=torch.int32), stream=0)
    assert (g.tokens, g.slots, g.struct.tokens) == (3, 6, 3)
    k._lib.result = result
    with pytest.raises(type(result) if isinstance(result, BaseException) else k.K3Error):
        g.plan(torch.zeros(8, 2, dtype=torch.int32), stream=0)
    assert (g.tokens, g.slots, g.struct.tokens) == (3, 6, 3)
    k._lib.result = 0
    g.plan(torch.zeros(5, 2, dtype=torch.int32), stream=0)
    assert (g.tokens, g.slots, g.struct.tokens) == (5, 10, 5)
