"""The plan of a routed batch against a stable sort, and the combine with its
gradients against fp64, over sizes, dropped and repeated ids, strides, types, in
place, order and capture."""
import numpy as np
import pytest
import torch

import e4m3_reference as ref
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _ids(T, kk, E, seed, kind="any"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, kk), E - 1, np.int32)
    if kind == "none":
        return rng.choice(np.array([-1, E, -7, 2 ** 31 - 1, -2 ** 31], np.int64), (T, kk)).astype(np.int32)
    ids = (E * rng.random((T, kk)) ** 2).astype(np.int32)  # some experts far more often; repeats in a token too
    if kind == "dropped":
        ids[rng.random((T, kk)) < 0.3] = -1
    return ids


def _check_plan(g, ids):
    want = ref.plan(ids, g.E)
    for got, w in zip((g.offsets, g.order, g.pos), want):
        assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("kind", ["any", "one", "none", "dropped"])
@pytest.mark.parametrize("T,kk,E", [(1, 1, 1), (1, 16, 896), (7, 3, 5), (64, 16, 128), (31, 32, 1024), (256, 32, 1000),
                                    (4096, 1, 33), (8192, 1, 1024), (2049, 2, 40), (4097, 1, 7), (4096, 16, 896), (20001, 5, 64),
                                    (8192, 16, 300), (8193, 16, 1024), (40001, 16, 300)])
def test_plan(T, kk, E, kind):
    ids = _ids(T, kk, E, T + E, kind)
    g = k.ExpertGroups(E, kk, T + 3)
    for t in (g.offsets, g._order, g._pos):
        t.fill_(-77)
    g.plan(torch.from_numpy(ids).cuda())
    _check_plan(g, ids)
    assert bool((g._order[T * kk:] == -77).all()) and bool((g._pos[T * kk:] == -77).all())
    small = ids[:max(1, T // 3)]  # another batch with the same object
    g.plan(torch.from_numpy(small).cuda())
    _check_plan(g, small)


def _case(T, kk, E, n, dt, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    ids = _ids(T, kk, E, seed, "dropped")
    g = k.ExpertGroups(E, kk, T)
    g.plan(torch.from_numpy(ids).cuda())
    y = torch.randn(T * kk, n + pad, generator=gen).to(DT[dt]).cuda()[:, :n]
    dout = torch.randn(T, n + 2 * pad, generator=gen).to(DT[dt]).cuda()[:, :n]
    w = torch.rand(T, kk, generator=gen).cuda()
    return g, ids, y, dout, w


def _gathered(ids, E, y):
    """[T][k][n] rows of each slot in fp64, zeros where dropped."""
    _, _, pos = ref.plan(ids, E)
    Y = np.zeros((ids.size, y.shape[1]))
    Y[pos >= 0] = y.double().cpu().numpy()[pos[pos >= 0]]
    return Y.reshape(*ids.shape, -1), pos.reshape(ids.shape)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,kk,E,n,pad", [(1, 1, 1, 1, 0), (1, 16, 896, 7168, 0), (5, 3, 4, 31, 1), (64, 8, 16, 1000, 8),
                                          (33, 9, 7, 2049, 0), (3, 32, 64, 2048, 0), (700, 2, 3, 40, 0), (2, 17, 5, 9000, 8)])
def test_combine(T, kk, E, n, pad, dt):
    g, ids, y, dout, w = _case(T, kk, E, n, dt, T + n, pad)
    Y, pos = _gathered(ids, E, y)
    W, D = w.double().cpu().numpy(), dout.double().cpu().numpy()
    for ww in (w, None):
        WW = W if ww is not None else np.ones_like(W)
        for acc in (False, True):
            out = torch.full((T, n + 3), 0.5, dtype=DT[dt], device="cuda")
            k.combine(out[:, :n], y, g, ww, accumulate=acc)
            want = np.einsum("tkn,tk->tn", Y, WW) + (0.5 if acc else 0)
            mag = np.einsum("tkn,tk->tn", np.abs(Y), WW) + 0.5
            assert (np.abs(out[:, :n].double().cpu().numpy() - want) <= mag * (kk + 1) * 2.0 ** -24 + np.abs(want) * HALF[dt]).all()
            assert bool((out[:, n:] == 0.5).all())
        dy = torch.full((T * kk, n + 1), 9.0, dtype=DT[dt], device="cuda")
        dw = torch.full((T, kk), 9.0, device="cuda") if ww is not None else None
        k.combine_backward(dy[:, :n], dw, dout, y if dw is not None else None, g, ww)
        got, kept = dy.double().cpu().numpy(), int((pos >= 0).sum())
        want = np.full((T * kk, n + 1), 9.0)
        t, j = np.nonzero(pos >= 0)
        want[pos[t, j], :n] = WW[t, j][:, None] * D[t]
        assert (np.abs(got - want) <= np.abs(want) * HALF[dt]).all()
        assert (got[kept:] == 9).all() and (got[:, n:] == 9).all()
        if dw is not None:
            want, mag = np.einsum("tkn,tn->tk", Y, D), np.einsum("tkn,tn->tk", np.abs(Y), np.abs(D))
            # a thread's terms one after the other (eight a step of 2048 columns), 5 + 8 joining steps
            terms = 8 * -(-n // (8 * min(256, -(-n // 256) * 32))) + 14
            assert (np.abs(dw.double().cpu().numpy() - want) <= mag * terms * 2.0 ** -24).all()
            assert bool((dw[torch.from_numpy(pos < 0).cuda()] == 0).all())


def test_gradients_against_differences():
    T, kk, E, n = 4, 3, 5, 40
    g, ids, y, dout, w = _case(T, kk, E, n, "f32", 9)
    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    k.combine_backward(dy, dw, dout, y, g, w)
    _, _, pos = ref.plan(ids, E)
    Y, W, D = y.double().cpu().numpy(), w.double().cpu().numpy(), dout.double().cpu().numpy()

    def f(Y, W):
        rows = np.where((pos >= 0)[:, None], Y[np.maximum(pos, 0)], 0.0).reshape(T, kk, n)
        return (np.einsum("tkn,tk->tn", rows, W) * D).sum()
    rng = np.random.default_rng(3)
    kept = (pos >= 0).sum()
    for _ in range(3):
        v, u = rng.standard_normal(Y.shape), rng.standard_normal(W.shape)
        v[kept:] = 0
        num = (f(Y + 1e-3 * v, W) - f(Y - 1e-3 * v, W)) / 2e-3  # linear in each: no error of the step
        assert abs((dy.double().cpu().numpy() * v).sum() - num) <= 1e-9 + 2.0 ** -20 * np.abs(dy.double().cpu().numpy() * v).sum()
        num = (f(Y, W + 1e-3 * u) - f(Y, W - 1e-3 * u)) / 2e-3
        assert abs((dw.double().cpu().numpy() * u).sum() - num) <= 1e-9 + 2.0 ** -20 * (np.abs(Y).sum() * np.abs(D).max())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_in_place_repeats_capture_and_other_stream(dt):
    T, kk, E, n = 300, 4, 9, 520
    g, ids, y, dout, w = _case(T, kk, E, n, dt, 12)
    t_ids = torch.from_numpy(ids).cuda()

    def run(o, g):
        g.plan(t_ids)
        k.combine(o[0], y, g, w)
        k.combine_backward(o[1], o[2], dout, y, g, w)

    def outs():
        return [torch.empty(T, n, dtype=DT[dt], device="cuda"), torch.zeros_like(y), torch.empty_like(w)]
    a, b, c = outs(), outs(), outs()
    run(a, g)
    over = y.clone()
    dw = torch.empty_like(w)
    k.combine_backward(over, dw, dout, over, g, w)
    kept = int(g.offsets[E])
    assert torch.equal(over[:kept], a[1][:kept]) and torch.equal(over[kept:], y[kept:]) and torch.equal(dw, a[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(b, k.ExpertGroups(E, kk, T))
    own = k.ExpertGroups(E, kk, T)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, own)
    t_ids.copy_(t_ids.flip(0))  # the graph reads its inputs anew
    graph.replay()
    torch.cuda.synchronize()
    _check_plan(own, t_ids.cpu().numpy())
    t_ids.copy_(t_ids.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    for p, q in zip(a, c):
        assert torch.equal(p, q)


def test_places_outside_the_rows_are_dropped():
    """A plan that a caller has damaged reads and writes no other memory."""
    T, kk, n = 6, 2, 64
    g, ids, y, dout, w = _case(T, kk, 3, n, "f32", 8)
    g._pos[0], g._pos[3], g._pos[5] = T * kk, -5, 2 ** 31 - 1
    out, dy, dw = torch.empty(T, n, device="cuda"), torch.zeros_like(y), torch.empty_like(w)
    k.combine(out, y, g, w)
    k.combine_backward(dy, dw, dout, y, g, w)
    pos = g.pos.cpu().numpy().reshape(T, kk)
    ok = (pos >= 0) & (pos < T * kk)
    Y = np.where(ok[..., None], y.double().cpu().numpy()[np.where(ok, pos, 0)], 0.0)
    want = np.einsum("tkn,tk->tn", Y, w.double().cpu().numpy())
    assert np.abs(out.double().cpu().numpy() - want).max() <= 1e-5
    assert bool((dw.cpu()[torch.from_numpy(~ok)] == 0).all())
