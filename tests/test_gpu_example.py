"""examples/train_expert.py: the operators together, a few steps."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu


def test_train_expert_learns_and_balances():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_expert
    losses, balances, counts, (y, z) = train_expert.train(steps=80)
    assert losses[-1] < 0.7 * losses[0]
    assert balances[-1] - 1 < 0.5 * (balances[0] - 1)
    assert int(counts.sum()) == 512 * 4
    # the packed expert's exact activations against the step's quantised ones:
    # MXFP4 rounding of x and h, about a tenth of an output vector
    assert float((y - z).norm() / y.norm()) < 0.3
    torch.cuda.synchronize()
    assert k.device_error() == 0
