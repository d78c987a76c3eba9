"""The balance loss over logits of any finite size, in place on rows that are not made
of aligned 16-byte units, and over more rows than the grids hold at once."""
import pytest
import torch

import test_gpu_balance as base
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT, RULES, ALPHA = base.DT, base.RULES, base.ALPHA


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


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("T,E,K", [(40, 33, 6), (5000, 33, 4), (5000, 64, 4)])
def test_in_place(T, E, K, rule):
    """dlogits on top of logits gives what separate ones give, rows loaded directly
    (33 experts) or copied ahead (64), with repeated ids."""
    l, ids, mask, w, dw = base.make(T, E, K, rule, "f32", 15, masked=0.2)
    ids[:, 3] = ids[:, 1]
    want = base.call(l, ids, mask, rule, 1.0, w, dw)
    bal, d = k.BalanceLoss(E, K, ALPHA, rule), torch.ones(1, device="cuda")
    for _ in range(3):
        x = l.clone()
        bal.backward(x, x, ids, want[1], want[2], d, mask, w, dw)
        assert torch.equal(x, want[3])


def test_mask_of_bools():
    l, ids, mask, w, dw = base.make(70, 48, 4, "softmax", "f32", 8, masked=0.4)
    for a, b in zip(base.call(l, ids, mask, "softmax", 1.0, w, dw), base.call(l, ids, mask.bool(), "softmax", 1.0, w, dw)):
        assert torch.equal(a, b)


# A pass of the forward grid covers 20 rows on each of 152 SMs (3040), one of the
# backward grid 3 x 8 (3648): these go round both loops, up to seven times, with
# rows in aligned 16-byte units (copied ahead) and without (loaded directly).
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("T,E,K,pad", [(3041, 8, 2, 0), (3649, 33, 4, 2), (7000, 256, 6, 0), (7000, 257, 6, 0),
                                       (20000, 64, 4, 0), (20011, 50, 3, 1), (8000, 896, 8, 0)])
def test_many_rows_a_warp(T, E, K, pad, rule, dt):
    l, ids, mask, w, dw = base.make(T, E, K, rule, dt, T + E, 0.3, 0.1, True, 0.02, pad)
    # whole runs of rows off, across the passes of both grids
    mask[3000:3700] = 0
    mask[6000:6200] = 0
    mask[-1] = 1
    got = base.call(l, ids, mask, rule, 1.5, w, dw)
    base.compare(l, ids, mask, rule, 1.5, w, dw, got)
    for a, b in zip(got, base.call(l, ids, mask, rule, 1.5, w, dw)):
        assert torch.equal(a, b)
