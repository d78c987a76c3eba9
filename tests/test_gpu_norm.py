"""8-bit rows and the norm: forward against fp64, its 8-bit rows code for code,
gradients against the formula and against differences; sizes from one, odd sizes,
strides, in place, extreme and non-finite rows, order and capture."""
import numpy as np
import pytest
import torch

import e4m3_reference as ref
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
# Of y = r s gain before the last rounding.  The sum of squares: a thread adds up to
# 64 terms one after the other, then 5 + 5 joining steps and one for its own square,
# all positive: (64 + 11) 2^-24, halved by the root.  1 / root within 2 ulp (2 * 2^-23),
# mean and eps 2 roundings (halved), two products.
REL = (38 + 4 + 1 + 2) * 2.0 ** -24


def _t(gen, T, n, dt, scale=1.0, pad=0):
    return (torch.randn(T, n + pad, generator=gen) * scale).to(DT[dt]).cuda()[:, :n]


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _stream(x, delta, dt):
    """r, from the fp32 sum (one rounding in fp32 rows, two in bf16's own type: the
    fp32 sum of two bf16 values rounds again only below 2^-16 of the larger)."""
    return x if delta is None else (x.float() + delta.float()).to(DT[dt])


def _formula(r, gain, eps):
    s = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    return r * s * (1 if gain is None else gain), s


CASES = [(1, 1, 0), (1, 7168, 0), (3, 31, 1), (5, 129, 0), (33, 1000, 8), (257, 1537, 0), (9, 1024, 0), (2, 8193, 0),
         (3, 8192, 8), (2, 16390, 0), (1, 32768, 0), (2, 32767, 1), (700, 64, 0), (2000, 40, 0),
         (700, 4099, 0), (400, 16392, 0), (330, 32765, 3)]  # the last three: several rows to a CTA that reads them twice


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,n,pad", CASES)
def test_forward(T, n, pad, dt):
    g = torch.Generator().manual_seed(T * 7 + n)
    x, delta = _t(g, T, n, dt, 3.0, pad), _t(g, T, n, dt, 1.0, 2 * pad)
    gain = (1 + torch.randn(n, generator=g) * 0.3).cuda()
    norm = k.RmsNorm(n, 1e-6)
    for d, gn in ((delta, gain), (None, gain), (delta, None)):
        y = torch.full((T, n + 3), 9.0, dtype=DT[dt], device="cuda")
        r = torch.full((T, n + 5), 9.0, dtype=DT[dt], device="cuda")
        rstd, y8 = torch.empty(T, device="cuda"), k.Mx8Rows(T, n)
        y8.codes.fill_(255), y8.scales.fill_(255)
        norm.forward(y[:, :n], x, d, r[:, :n] if d is not None else None, rstd, gn, y8)
        want_r = _stream(x, d, dt)
        if d is not None:
            assert torch.equal(r[:, :n], want_r) and bool((r[:, n:] == 9).all())
        want, s = _formula(_f64(want_r), _f64(gn), np.float32(1e-6))
        assert (np.abs(_f64(y[:, :n]) - want) <= np.abs(want) * (REL + HALF[dt]) + 1e-38).all()
        assert bool((y[:, n:] == 9).all())
        assert (np.abs(_f64(rstd)[:, None] - s) <= s * REL).all()
        got, scales, clean = ref.read_rows(y8)
        assert clean, "bytes past the rows"
        if dt == "f32":  # y is what was quantised
            v, e = ref.quantize(y[:, :n].cpu().numpy())
            assert np.array_equal(scales, e) and np.array_equal(got, v)
        else:  # within the rounding of e4m3 (2^-4, or half the smallest step at the scale)
            # and what y before its rounding is off; a scale at its border may be the next
            step = np.repeat(np.ldexp(1.0, scales - 127), 32, axis=1)[:, :n] * 2.0 ** -10
            assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 2 * REL) + step).all()
            v, e = ref.quantize(want.astype(np.float32))
            assert (np.abs(scales - e) <= 1).all() and (got != v).mean() <= 1e-3


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,n,pad", CASES)
def test_backward(T, n, pad, dt):
    g = torch.Generator().manual_seed(T * 5 + n)
    r, dy, dr = _t(g, T, n, dt, 2.0, pad), _t(g, T, n, dt, 1.0, 2 * pad), _t(g, T, n, dt, 0.5, pad)
    gain = (1 + torch.randn(n, generator=g) * 0.3).cuda()
    norm = k.RmsNorm(n, 1e-5)
    rstd, y = torch.empty(T, device="cuda"), torch.empty(T, n, dtype=DT[dt], device="cuda")
    norm.forward(y, r, rstd=rstd, gain=gain)
    R, S, DY, DR, G = _f64(r), _f64(rstd)[:, None], _f64(dy), _f64(dr), _f64(gain)
    for res, gn in ((dr, gain), (None, gain), (dr, None)):
        dx = torch.full((T, n + 1), 9.0, dtype=DT[dt], device="cuda")
        dgain = torch.full((n,), 5.0, device="cuda")
        norm.backward(dx[:, :n], dgain if gn is not None else None, dy, r, rstd, gn, res)
        gg, xh = DY * (G if gn is not None else 1), R * S
        dot = (gg * xh).mean(1, keepdims=True)
        want = S * (gg - xh * dot) + (DR if res is not None else 0)
        # the dot product's sum: 64 terms in a thread and 11 joining steps, each of two
        # products; then four more roundings of the parts before they cancel
        mag = S * (np.abs(gg) + np.abs(xh) * ((np.abs(gg * xh)).mean(1, keepdims=True) * 78 + np.abs(dot)))
        tol = (mag * 6 + (np.abs(DR) if res is not None else 0)) * 2.0 ** -24 + np.abs(want) * HALF[dt] + 1e-38
        assert (np.abs(_f64(dx[:, :n]) - want) <= tol).all()
        assert bool((dx[:, n:] == 9).all())
        if gn is None:
            continue
        # column sums: a team's rows one after the other, then up to 64 parts a warp and 8
        # warps; two products a term
        rows = -(-T // min(512, T)) + 64 + 8 + 2
        want_g, mag = (DY * xh).sum(0), np.abs(DY * xh).sum(0)
        assert (np.abs(_f64(dgain) - want_g) <= mag * rows * 2.0 ** -24 + 1e-38).all()
        before = dgain.clone()
        norm.backward(dx[:, :n], dgain, dy, r, rstd, gn, res, accumulate=True)
        assert torch.equal(dgain, before + before)


def test_gradients_against_differences():
    """Directional differences of <dy, y> + <dr, r> over x, and over gain, of the fp64
    formula at the kernel's inputs."""
    T, n, eps = 3, 96, 1e-3
    g = torch.Generator().manual_seed(2)
    r, dy, dr = (_t(g, T, n, "f32") for _ in range(3))
    gain = (1 + torch.randn(n, generator=g) * 0.3).cuda()
    norm = k.RmsNorm(n, eps)
    rstd, y, dx, dgain = torch.empty(T, device="cuda"), torch.empty_like(r), torch.empty_like(r), torch.empty(n, device="cuda")
    norm.forward(y, r, rstd=rstd, gain=gain)
    norm.backward(dx, dgain, dy, r, rstd, gain, dr)
    R, G, DY, DR, h = _f64(r), _f64(gain), _f64(dy), _f64(dr), 1e-5
    f = lambda R, G: (DY * _formula(R, G, np.float32(eps))[0]).sum() + (DR * R).sum()  # noqa: E731
    rng = np.random.default_rng(1)
    for _ in range(4):
        v, w = rng.standard_normal(R.shape), rng.standard_normal(G.shape)
        num = (f(R + h * v, G) - f(R - h * v, G)) / (2 * h)
        # h^2 times the third derivative (below 100 here), and the fp32 gradients' own error
        assert abs((_f64(dx) * v).sum() - num) <= 1e-7 + 1e-4 * np.abs(_f64(dx) * v).sum() * 2 ** -7
        num = (f(R, G + h * w) - f(R, G - h * w)) / (2 * h)
        assert abs((_f64(dgain) * w).sum() - num) <= 1e-7 + 1e-4 * np.abs(_f64(dgain) * w).sum() * 2 ** -7


@pytest.mark.parametrize("n", [8, 100, 7168, 4099, 20000])
def test_rows_out_of_range(n):
    """Zeros, rows whose squares leave fp32 both ways, infinities and NaN; each row by
    itself, eps 0 and 1e-6."""
    g = torch.Generator().manual_seed(n)
    base = torch.randn(1, n, generator=g).clamp(-3, 3)
    scales = [0.0, 1e-30, 1e-25, 1e-18, 1.0, 1e19, 1e30, 1e37]
    x = torch.cat([base * s for s in scales] + [base.clone(), base.clone(), base.clone()])
    x[-3, n // 2], x[-2, 0], x[-1, n - 1] = float("nan"), float("inf"), 3e38
    for eps in (0.0, 1e-6):
        y, y8, rstd = torch.empty(x.shape, device="cuda"), k.Mx8Rows(x.shape[0], n), torch.empty(x.shape[0], device="cuda")
        k.RmsNorm(n, eps).forward(y, x.cuda(), rstd=rstd, y8=y8)
        X = x.numpy().astype(np.float64)
        with np.errstate(all="ignore"):
            want, s = _formula(X, None, np.float32(eps))
        got, got_s = _f64(y), _f64(rstd)
        for i in [j for j in range(len(scales)) if eps or scales[j]] + [-1]:
            # values or their root below fp32's normal numbers lose more than a rounding
            ok = np.abs(X[i]) > 1e-36
            assert (np.abs(got[i] - want[i]) <= np.abs(want[i]) * (REL + 2.0 ** -24) + 1e-37)[ok].all(), (eps, i)
            assert abs(got_s[i] - s[i, 0]) <= s[i, 0] * REL, (eps, i)
        if not eps:
            assert np.isnan(got[0]).all()  # 0 / 0
        assert np.isnan(got[-3]).all()
        rest = np.delete(got[-2], 0)
        assert np.isnan(got[-2, 0]) and not rest.any()  # finite / infinity
        v, sc, _ = ref.read_rows(y8)
        e = ref.quantize(y.cpu().numpy())
        assert np.array_equal(v, e[0], equal_nan=True) and np.array_equal(sc, e[1])


@pytest.mark.parametrize("T,n", [(50, 200), (400, 4100), (400, 16640)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_in_place(dt, T, n):
    g = torch.Generator().manual_seed(4)
    x, d, dy, dr = (_t(g, T, n, dt) for _ in range(4))
    gain = torch.rand(n, generator=g).cuda()
    norm = k.RmsNorm(n, 1e-6)
    y, r, rstd, dx = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty_like(x)
    norm.forward(y, x, d, r, rstd, gain)
    for to_x in (True, False):
        a, b = x.clone(), d.clone()
        norm.forward(b if to_x else a, a, b, a if to_x else b, None, gain)  # r over one, y over the other
        assert torch.equal(a, r if to_x else y) and torch.equal(b, y if to_x else r)
    norm.backward(dx, None, dy, r, rstd, gain, dr)
    for which in range(3):
        v = [dy.clone(), dr.clone(), r.clone()]
        norm.backward(v[which], None, v[0], v[2], rstd, gain, v[1])
        assert torch.equal(v[which], dx)


@pytest.mark.parametrize("n", [1024, 1001])
def test_gains_of_any_alignment(n):
    g = torch.Generator().manual_seed(n)
    x, dy = _t(g, 9, n, "bf16"), _t(g, 9, n, "bf16")
    gains = torch.rand(n + 1, generator=g).cuda()
    norm, outs = k.RmsNorm(n, 1e-6), []
    for gain in (gains[1:], gains[1:].clone()):
        y, dx, rstd, dgain = torch.empty_like(x), torch.empty_like(x), torch.empty(9, device="cuda"), torch.empty(n + 1, device="cuda")
        norm.forward(y, x, None, None, rstd, gain)
        norm.backward(dx, dgain[1:], dy, x, rstd, gain)
        outs.append((y, dx, dgain[1:].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_repeats_capture_and_other_stream(dt):
    T, n = 1500, 264
    g = torch.Generator().manual_seed(5)
    x, d, dy = (_t(g, T, n, dt) for _ in range(3))
    gain = torch.rand(n, generator=g).cuda()

    def run(o, norm):
        norm.forward(o[0], x, d, o[1], o[2], gain, o[5])
        norm.backward(o[3], o[4], dy, o[1], o[2], gain, dy)

    def outs():
        return [torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty_like(x),
                torch.empty(n, device="cuda"), k.Mx8Rows(T, n)]

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a[:5], b[:5])) and torch.equal(a[5].codes, b[5].codes) and \
            torch.equal(a[5].scales, b[5].scales)
    a, b, c = outs(), outs(), outs()
    run(a, k.RmsNorm(n, 1e-6))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(b, k.RmsNorm(n, 1e-6))
    norm = k.RmsNorm(n, 1e-6)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, norm)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(a, b) and same(a, c)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,n,pad", [(1, 1, 0), (1, 31, 0), (3, 33, 1), (5, 128, 0), (17, 129, 3), (40, 1000, 8),
                                     (2, 7168, 0), (333, 260, 4), (1, 70000, 0), (1000, 100, 0)])
def test_rows_in_8_bits(T, n, pad, dt):
    g = torch.Generator().manual_seed(n)
    x = _t(g, T, n, dt, 1.0, pad) * torch.exp2(torch.randint(-9, 9, (T, 1), generator=g).float()).cuda().to(DT[dt])
    x = torch.nn.functional.pad(x, (0, pad))[:, :n]
    o = k.Mx8Rows(T, n)
    o.codes.fill_(255), o.scales.fill_(255)
    k.mx8_quantize(o, x)
    v, s = ref.quantize(x.float().cpu().numpy())
    got, scales, clean = ref.read_rows(o)
    assert clean and np.array_equal(scales, s) and np.array_equal(got, v)
    y = torch.full((T, n + pad), 7.0, dtype=DT[dt], device="cuda")
    k.mx8_dequantize(y[:, :n], o)
    assert np.array_equal(_f64(y[:, :n]), v) and bool((y[:, n:] == 7).all())


def test_rows_in_8_bits_at_the_edges():
    """Scales at the 448 border, ties, zeros, subnormals, the largest and non-finite
    values, each a block of one row."""
    blocks = [np.full(32, 448.0), np.full(32, 448.00003), np.linspace(-1.75, 1.75, 32), np.linspace(-1.7500001, 1.75, 32),
              np.zeros(32), 1e-40 * np.arange(32), np.linspace(-3.4e38, 3.4e38, 32), np.linspace(-100, 100, 32),
              TABLE_TIES(), np.where(np.arange(32) == 5, np.inf, 1.0), np.where(np.arange(32) == 31, np.nan, 2.0), -np.zeros(32)]
    x = np.concatenate(blocks).astype(np.float32)[None]
    o = k.Mx8Rows(1, x.shape[1])
    k.mx8_quantize(o, torch.from_numpy(x).cuda())
    v, s = ref.quantize(x)
    got, scales, clean = ref.read_rows(o)
    assert clean and np.array_equal(scales, s) and np.array_equal(got, v, equal_nan=True)
    y = torch.empty(x.shape, device="cuda")
    k.mx8_dequantize(y, o)
    assert np.array_equal(_f64(y), v, equal_nan=True)


def TABLE_TIES():
    t = (ref.TABLE[10:42] + ref.TABLE[11:43]) / 2
    t[-1] = 448.0  # scale 1
    return t
