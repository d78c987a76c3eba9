"""Every form of the grouped product over lengths of K that end inside and before its
pipeline, odd widths, row strides and places of C; the form that runs is asserted.  Against
fp64 products of the values that the rows and matrices stand for."""
import functools

import numpy as np
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k
from test_gpu_grouped import DT, HALF, _plan, _rows, _sources, _wide

pytestmark = pytest.mark.gpu

# Groups that run in each form at 9000 columns, none and one row among them, ends inside and
# at a tile; pairs with one tile a group and with several.
SIZES = {"16": [0, 1, 16, 17, 5, 9], "32": [33, 0, 31, 1, 15, 16], "64": [64, 65, 0, 1, 50, 36],
         "pairs": [256, 0, 1, 140, 133, 31], "tiles": [300, 257, 31, 0, 513, 95]}
ROWS = {"16": 16, "32": 32, "64": 64, "pairs": 256, "tiles": 256}
# 1, 2, 3, 5, 7, 9 and 10 steps of 128: fewer than the stages, fewer than a ring of tiles has
# them, scale bytes of four steps at a time with a rest of 1, 2 and 3
LENGTHS = [128, 256, 384, 640, 896, 1152, 1280]
# (tiles of 64 rows are chosen from five steps on)
CASES = [(form, K) for form in SIZES for K in LENGTHS if form != "64" or K >= 640]


@functools.lru_cache(maxsize=1)
def _matrices(N, K):
    return _wide(6, N, K)


def _check(N, K, form, gather, out, pad, at, accumulate=False):
    """C: N columns from column `at` of rows that are `pad` wider."""
    W, V = _matrices(N, K)
    E, sizes = 6, SIZES[form]
    assert k.grouped_matmul_form(E, sum(sizes), N, K) == ROWS[form]
    g, ids = _plan(sizes, 1, 5)
    a, A = _rows(ids.size, K, 3)
    off, src = _sources(ids, E, gather)
    A = torch.from_numpy(A).cuda()[torch.from_numpy(np.ascontiguousarray(src)).cuda()]

    def run():
        whole = torch.full((ids.size, N + pad), 0.5, dtype=DT[out], device="cuda")
        k.grouped_matmul(whole[:, at:at + N], a, W, g, gather=gather, accumulate=accumulate)
        return whole
    whole = run()
    C = whole[:, at:at + N]
    assert bool((whole[:, :at] == 0.5).all()) and bool((whole[:, at + N:] == 0.5).all())
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        want, mag = A[s] @ V[e].t(), A[s].abs() @ V[e].abs().t()
        if accumulate:
            want, mag = want + 0.5, mag + 0.5
        # 2^-22 of the magnitudes for each 32 columns of K and a few more, as in the tests of
        # one width
        tol = mag * (K / 32 + 10) * 2.0 ** -22 + want.abs() * HALF[out]
        assert bool(((C[s].double() - want).abs() <= tol).all()), e
    assert bool((C[int(off[E]):] == 0.5).all())
    assert torch.equal(run(), whole) and k.device_error() == 0


@pytest.mark.parametrize("out,acc", [("f32", False), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("form,K", sorted(CASES, key=lambda c: c[1]))
def test_odd_width(form, K, gather, out, acc):
    """An odd number of columns in rows of an odd stride: single stores in both types."""
    _check(9001, K, form, gather, out, 6, 3, acc)


@pytest.mark.parametrize("N,pad,at", [(9000, 4, 2), (9000, 4, 1), (9000, 5, 2), (8999, 1, 0)])
@pytest.mark.parametrize("form", list(SIZES))
def test_columns_in_pairs_or_not(form, N, pad, at):
    """bf16 results whose columns can and cannot be stored two at a time: by address, by
    stride and by width."""
    _check(N, 640, form, True, "bf16", pad, at)
