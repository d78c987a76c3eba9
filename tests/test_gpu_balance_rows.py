"""The balance loss over logits of any finite size."""
import pytest
import torch

import test_gpu_balance as base

pytestmark = pytest.mark.gpu
DT, RULES = base.DT, base.RULES


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("level", ["low", -1e30, -1e10, -3e9, 3e9, 1e10, 1e30, "high"])
@pytest.mark.parametrize("E", [72, 33])
def test_rows_of_large_logits(E, level, rule, dt):
    """Rows wholly at one large value (every expert of a token masked by a finite
    number: p = 1/E) or about one, between ordinary rows and rows in which some
    experts are at that value."""
    l, ids, _, w, dw = base.make(40, E, 5, rule, dt, E)
    at = {"low": torch.finfo(DT[dt]).min, "high": torch.finfo(DT[dt]).max}.get(level, level)
    l = l.contiguous()
    l[3] = at
    l[11] = at
    l[12] = l[12] * abs(at) * 0.01 if abs(at) < 1e36 else at
    l[20, ::3] = -abs(at)
    l[21:30, 5] = -abs(at)
    base.compare(l, ids, None, rule, 1.5, w, dw, base.call(l, ids, None, rule, 1.5, w, dw))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rule", RULES)
def test_only_rows_at_the_lowest_value(rule, dt):
    l, ids, _, w, dw = base.make(9, 48, 4, rule, dt, 2)
    l = torch.full_like(l, torch.finfo(DT[dt]).min)
    got = base.call(l, ids, None, rule, 1.0, w, dw)
    base.compare(l, ids, None, rule, 1.0, w, dw, got)
    assert int(got[2]) == 9 and bool(torch.isfinite(got[3]).all())
