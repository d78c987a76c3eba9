"""SwiGLU with its 8-bit checkpoint: the forward output, the kept values bit for
bit, and the gradients from them against fp64 formulas and against differences,
over sizes, strides, types and non-finite blocks."""
import numpy as np
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}

TABLE = np.array([m * 2.0 ** -9 for m in range(8)] +
                 [(8 + m) * 2.0 ** (p - 3) for p in range(-6, 9) for m in range(8)][:119])  # 0 .. 448


def kept(x):
    """(values, scale bytes) of the checkpoint of x [T][f] (fp64 from fp32)."""
    T, f = x.shape
    pad = -(-f // 32) * 32
    v = np.zeros((T, pad))
    v[:, :f] = x
    v = v.reshape(T, pad // 32, 32)
    top = np.abs(v).max(-1)
    finite = np.isfinite(v).all(-1)
    e = np.zeros(top.shape, np.int64)
    for i in np.ndindex(*top.shape):
        if finite[i] and top[i] > 0:
            e[i] = max(next(b for b in range(int(np.floor(np.log2(top[i]))) + 118 - 2, 300)
                            if top[i] <= 448 * 2.0 ** (b - 127)), 0)
    a = np.abs(np.where(finite[..., None], v, 0.0)) * np.ldexp(1.0, 127 - e)[..., None]
    lo = np.clip(np.searchsorted(TABLE, a, side="right") - 1, 0, TABLE.size - 1)
    hi = np.minimum(lo + 1, TABLE.size - 1)
    d = (a - TABLE[lo]) - (TABLE[hi] - a)
    up = (d > 0) | ((d == 0) & (lo % 2 == 1))
    q = TABLE[np.where(up & (hi > lo), hi, lo)] * np.ldexp(1.0, e - 127)[..., None]
    q = np.where(np.signbit(v), -q, q)
    q = np.clip(q, -240 * 2.0 ** 120, 240 * 2.0 ** 120)  # a finite value reads back finite
    q[~finite] = np.nan
    return q.reshape(T, pad)[:, :f], np.where(finite, e, 255)


def _inputs(T, f, dt, seed, fused=False, pad=0):
    g = torch.Generator().manual_seed(seed)

    def one(n, s):
        return (torch.randn(T, n, generator=g) * s).to(DT[dt]).cuda()
    if fused:
        gu = one(2 * f + pad, 2.0)
        return gu[:, :f], gu[:, f:2 * f], one(f, 0.1)
    return one(f + pad, 2.0)[:, :f], one(f + pad, 1.0)[:, :f], one(f + pad, 0.1)[:, :f]


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _sigma(g):
    return 1.0 / (1.0 + np.exp(-g))


def _check_ckpt(ck, g, u):
    T, f = g.shape
    pad = -(-f // 32) * 32
    b = ck.data.cpu().numpy()
    codes, scales = b[:2 * T * pad].reshape(2, T, pad), b[2 * T * pad:2 * T * pad + 2 * T * pad // 32]
    scales = scales.reshape(2, T, pad // 32)
    out = []
    for i, x in enumerate((g, u)):
        want, e = kept(x)
        assert np.array_equal(scales[i], e)
        c = codes[i]
        got = np.where(c & 128, -1.0, 1.0) * TABLE[np.minimum(c & 127, 126)]
        got = got * np.repeat(np.ldexp(1.0, scales[i].astype(np.int64) - 127), 32, axis=1)
        fin = np.repeat(scales[i] != 255, 32, axis=1)
        assert np.array_equal(got[:, :f][fin[:, :f]], want[fin[:, :f]]), "kept values"
        assert not codes[i][:, f:].any(), "codes past f"
        out.append(want)
    return out


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,f,fused,pad", [(1, 1, False, 0), (1, 1536, False, 0), (3, 31, True, 0), (5, 32, False, 1),
                                           (17, 100, True, 0), (64, 257, False, 3), (40, 1000, True, 8),
                                           (2, 4096, False, 8)])
def test_forward_backward(T, f, fused, pad, dt):
    g, u, dh = _inputs(T, f, dt, T + f, fused, pad)
    h = torch.full((T, f + 2), 9.0, dtype=DT[dt], device="cuda")
    ck = k.SwigluCheckpoint(T, f)
    ck.data.fill_(255)
    k.swiglu_forward(h[:, :f], ck, g, u)
    dg, du = torch.empty(T, f, dtype=DT[dt], device="cuda"), torch.empty(T, f, dtype=DT[dt], device="cuda")
    k.swiglu_backward(dg, du, dh, ck)
    torch.cuda.synchronize()
    G, U, D = _f64(g), _f64(u), _f64(dh)
    # sigma: exp and a division within 3 ulp each, then two products
    rel = 10 * 2.0 ** -24
    want = G * _sigma(G) * U
    assert (np.abs(_f64(h[:, :f]) - want) <= np.abs(want) * (rel + HALF[dt]) + 1e-38).all()
    assert bool((h[:, f:] == 9).all())
    G, U = _check_ckpt(ck, G, U)
    s = _sigma(G)
    want_u = D * G * s
    assert (np.abs(_f64(du) - want_u) <= np.abs(want_u) * (rel + HALF[dt]) + 1e-38).all()
    want_g = D * U * s * (1 + G * (1 - s))
    # 1 - sigma and the sum with 1 lose 2^-24 of their own size before they cancel
    slack = np.abs(D * U * s) * (1 + 2 * np.abs(G)) * rel
    assert (np.abs(_f64(dg) - want_g) <= slack + np.abs(want_g) * HALF[dt] + 1e-38).all()


def test_gradients_against_differences():
    """dg and du of one row against central differences of <dh, silu(g) u> at
    the kept values."""
    T, f = 2, 48
    g, u, dh = _inputs(T, f, "f32", 77)
    ck = k.SwigluCheckpoint(T, f)
    h, dg, du = (torch.empty(T, f, device="cuda") for _ in range(3))
    k.swiglu_forward(h, ck, g, u)
    k.swiglu_backward(dg, du, dh, ck)
    G, U, D = kept(_f64(g))[0], kept(_f64(u))[0], _f64(dh)
    e = 1e-5

    def part(G, U):
        return D * G * _sigma(G) * U
    num_g = (part(G + e, U) - part(G - e, U)) / (2 * e)
    num_u = (part(G, U + e) - part(G, U - e)) / (2 * e)
    # e^2 / 6 times the third derivative (below 1 per unit of dh u), and the fp32 result
    assert np.abs(_f64(dg) - num_g).max() <= 1e-9 + 1e-6 * np.abs(D * U * (1 + np.abs(G))).max()
    assert np.abs(_f64(du) - num_u).max() <= 1e-9 + 1e-6 * np.abs(D * G).max()


def test_checkpoint_edges():
    """Scales at the 448 border, zeros, subnormals, the largest and non-finite
    values; saturated gates."""
    rows = [np.full(32, 448.0), np.full(32, 448.00003), np.linspace(-1.75, 1.75, 32), np.linspace(-1.7500001, 1.75, 32),
            np.zeros(32), 1e-40 * np.arange(32), np.linspace(-3.4e38, 3.4e38, 32), np.linspace(-100, 100, 32),
            TABLE[:32] * 2.0 ** -9, (TABLE[10:42] + TABLE[11:43]) / 2]
    x = np.stack(rows).astype(np.float32)
    x[-2, -1] = 448.0  # scale 1: the entries below are exact or subnormal
    x[-1, -1] = 448.0
    ones = np.ones_like(x)
    ck = k.SwigluCheckpoint(*x.shape)
    h = torch.empty(x.shape, device="cuda")
    k.swiglu_forward(h, ck, torch.from_numpy(x).cuda(), torch.from_numpy(ones).cuda())
    _check_ckpt(ck, x.astype(np.float64), ones.astype(np.float64))
    dg, du = torch.empty_like(h), torch.empty_like(h)
    k.swiglu_backward(dg, du, torch.ones_like(h), ck)
    assert bool(torch.isfinite(dg).all()) and bool(torch.isfinite(du).all())


def test_nonfinite_block_shows_in_the_gradients():
    T, f = 3, 96
    g, u, dh = _inputs(T, f, "f32", 5)
    g[1, 40] = float("inf")
    u[2, 3] = float("nan")
    ck = k.SwigluCheckpoint(T, f)
    h, dg, du = (torch.empty(T, f, device="cuda") for _ in range(3))
    k.swiglu_forward(h, ck, g, u)
    k.swiglu_backward(dg, du, dh, ck)
    bad_g, bad_u = torch.zeros(T, f, dtype=torch.bool), torch.zeros(T, f, dtype=torch.bool)
    bad_g[1, 32:64] = bad_u[1, 32:64] = True   # g unknown: both gradients
    bad_g[2, :32] = True                        # u unknown: only dg uses it
    assert torch.equal(torch.isnan(dg).cpu(), bad_g)
    assert torch.equal(torch.isnan(du).cpu(), bad_u)


def test_backward_in_place_and_graph():
    T, f = 50, 200
    g, u, dh = _inputs(T, f, "bf16", 6)
    ck = k.SwigluCheckpoint(T, f)
    h, dg, du = (torch.empty(T, f, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    k.swiglu_forward(h, ck, g, u)
    k.swiglu_backward(dg, du, dh, ck)
    same, du2 = dh.clone(), torch.empty_like(du)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k.swiglu_forward(h, ck, g, u)
        k.swiglu_backward(same, du2, same, ck)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(same, dg) and torch.equal(du2, du)
