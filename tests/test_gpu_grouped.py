"""Products grouped by expert: 8-bit rows times MXFP4 matrices, and the weight
gradients, against fp64 products of the values they stand for, over group sizes from
none, odd sizes, tiles of every width, strides, both types, and bad values that must
stay in their rows."""
import numpy as np
import pytest
import torch

import e4m3_reference as ref
import mx_reference as mx
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _ids(sizes, kk, seed):
    """ids [T][kk] in mixed order with `sizes` slots for each expert, the rest dropped."""
    flat = np.concatenate([np.full(n, e, np.int32) for e, n in enumerate(sizes)])
    flat = np.concatenate([flat, np.full(-flat.size % kk, -1, np.int32)])
    np.random.default_rng(seed).shuffle(flat)
    return flat.reshape(-1, kk)


def _plan(sizes, kk, seed=0):
    ids = _ids(sizes, kk, seed)
    g = k.ExpertGroups(len(sizes), kk, ids.shape[0])
    g.plan(torch.from_numpy(ids).cuda())
    return g, ids


def _weights(E, N, K, seed, lo=120, hi=131):
    rng = np.random.default_rng(seed)
    packed = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi, (E, N, K // 32), dtype=np.uint8)
    W = k.MxExperts.from_matrices(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda())
    return W, np.stack([mx.values(mx.unpack(p), s) for p, s in zip(packed, scales)])


def _rows(rows, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-4, 5, (rows, 1), generator=g).float())
    a = k.Mx8Rows(rows, K)
    k.mx8_quantize(a, x.cuda())
    return a, ref.quantize(x.numpy())[0]


def _sources(ids, E, gather):
    off, order, _ = ref.plan(ids, E)
    return off, order[:off[E]] // ids.shape[1] if gather else np.arange(off[E])


def _want(off, src, A, V):
    """(product, its magnitudes) of the kept rows."""
    c, m = np.zeros((src.size, V.shape[1])), np.zeros((src.size, V.shape[1]))
    for e in range(V.shape[0]):
        s = slice(off[e], off[e + 1])
        c[s], m[s] = A[src[s]] @ V[e].T, np.abs(A[src[s]]) @ np.abs(V[e]).T
    return c, m


# group sizes for tiles of each width (16 rows and up by the average), none and one
# among them, ends inside and at a tile
SIZES = {"one": [1], "few": [0, 1, 3, 16, 17, 0, 5, 2], "some": [33, 0, 1, 32, 31, 7], "more": [65, 64, 1, 0, 40],
         "many": [200, 128, 129, 1, 0, 257], "single": [0, 0, 300, 0], "empty": [0, 0, 0]}


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("N,K,kk,pad", [(128, 128, 1, 2), (200, 384, 2, 0), (1, 1152, 3, 3), (129, 256, 4, 1),
                                        (1000, 640, 5, 3)])
def test_matmul(N, K, kk, pad, sizes, gather, out):
    sizes = SIZES[sizes]
    if not sum(sizes):
        g, ids = k.ExpertGroups(len(sizes), kk, 4), np.full((4, kk), -1, np.int32)
        g.plan(torch.from_numpy(ids).cuda())
    else:
        g, ids = _plan(sizes, kk)
    E, slots = len(sizes), ids.size
    W, V = _weights(E, N, K, N + K)
    a, A = _rows(ids.shape[0] if gather else slots, K, 3)
    C = torch.full((slots, N + pad), 9.0, dtype=DT[out], device="cuda")
    k.grouped_matmul(C[:, :N], a, W, g, gather=gather)
    off, src = _sources(ids, E, gather)
    want, mag = _want(off, src, A, V)
    kept = off[E]
    got = C.double().cpu().numpy()
    # an fp32 step (at most K / 32 and a few) loses 2^-22 of the sum of magnitudes, as in
    # the operands' product
    tol = mag * (K / 32 + 10) * 2.0 ** -22 + np.abs(want) * HALF[out]
    assert (np.abs(got[:kept, :N] - want) <= tol).all()
    assert (got[kept:] == 9).all() and (got[:, N:] == 9).all()
    again = torch.full_like(C, 9.0)
    k.grouped_matmul(again[:, :N], a, W, g, gather=gather)
    assert torch.equal(again, C)
    if out == "f32":
        k.grouped_matmul(C[:, :N], a, W, g, gather=gather, accumulate=True)
        assert bool((C[:kept, :N] == again[:kept, :N] + again[:kept, :N]).all()) and bool((C[kept:] == 9).all())
    assert k.device_error() == 0


@pytest.mark.parametrize("T,kk,E,N,K", [(1, 16, 896, 256, 1024), (64, 16, 128, 384, 512), (300, 8, 1024, 128, 256),
                                        (700, 16, 24, 512, 384)])
def test_matmul_many_experts(T, kk, E, N, K):
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:kk] for _ in range(T)]).astype(np.int32)
    g = k.ExpertGroups(E, kk, T)
    g.plan(torch.from_numpy(ids).cuda())
    W, V = _weights(E, N, K, 5)
    a, A = _rows(T, K, 4)
    C = torch.empty(T * kk, N, device="cuda")
    k.grouped_matmul(C, a, W, g, gather=True)
    off, src = _sources(ids, E, True)
    want, mag = _want(off, src, A, V)
    assert (np.abs(C.double().cpu().numpy() - want) <= mag * (K / 32 + 10) * 2.0 ** -22 + np.abs(want) * 2.0 ** -24).all()


def test_matmul_of_the_longest_rows():
    for K, sizes in ((1 << 20, [1, 20]), (1 << 17, [70, 100])):
        W, V = _wide(2, 8, K)
        _check_wide(W, V, sizes, 1, True, "f32")


def _wide(E, N, K):
    """Random stored matrices on the GPU and their fp64 values."""
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    packed = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(120, 131, (E, N, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    lut = torch.tensor(np.concatenate([mx.MAG, -mx.MAG]), device="cuda")
    V = torch.empty(E, N, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        V[e, :, 0::2], V[e, :, 1::2] = lut[(packed[e] & 15).long()], lut[(packed[e] >> 4).long()]
        V[e] *= torch.exp2(scales[e].double() - 127).repeat_interleave(32, 1)
    return k.MxExperts.from_matrices(packed, scales), V


def _check_wide(W, V, sizes, kk, gather, out, accumulate=False):
    E, N, K = V.shape
    g, ids = _plan(sizes, kk, 5)
    a, A = _rows(ids.shape[0] if gather else ids.size, K, 3)
    off, src = _sources(ids, E, gather)
    A = torch.from_numpy(A).cuda()[torch.from_numpy(src).cuda()]
    C = torch.full((ids.size, N), 0.5, dtype=DT[out], device="cuda")
    k.grouped_matmul(C, a, W, g, gather=gather, accumulate=accumulate)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        want, mag = A[s] @ V[e].t(), A[s].abs() @ V[e].abs().t()
        if accumulate:
            want, mag = want + 0.5, mag + 0.5
        tol = mag * (K / 32 + 10) * 2.0 ** -22 + want.abs() * HALF[out]
        assert bool(((C[s].double() - want).abs() <= tol).all()), e
    assert bool((C[off[E]:] == 0.5).all())
    again = torch.full_like(C, 0.5)
    k.grouped_matmul(again, a, W, g, gather=gather, accumulate=accumulate)
    assert torch.equal(again, C) and k.device_error() == 0


# by the form that runs: tiles of 16, 32 and 64 rows, and pairs of CTAs
FORMS = {16: [0, 1, 16, 17, 5, 9], 32: [33, 0, 31, 1, 15, 16], 64: [64, 65, 0, 1, 50, 36], 256: [256, 0, 1, 40, 33, 31]}


@pytest.fixture(scope="module")
def wide():
    return _wide(6, 9000, 1024)


@pytest.mark.parametrize("out,acc", [("f32", False), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("form", list(FORMS))
def test_matmul_every_form(wide, form, gather, out, acc):
    sizes = FORMS[form]
    assert k.grouped_matmul_form(6, sum(sizes), 9000, 1024) == form
    _check_wide(*wide, sizes, 1, gather, out, acc)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes", [[300, 257, 31, 0, 513, 95], [1025, 255, 256, 512, 2, 480]])
def test_matmul_pairs_of_several_tiles(wide, sizes, gather, out):
    assert k.grouped_matmul_form(6, sum(sizes), 9000, 1024) == 256
    _check_wide(*wide, sizes, 1, gather, out)


# few tiles of a long K: those left over from full waves are shared by several CTAs
@pytest.mark.parametrize("form,each", [(32, 16), (64, 40)])
def test_matmul_tiles_in_parts(form, each):
    W, V = _wide(80, 250, 4096)
    rng = np.random.default_rng(each)
    sizes = rng.integers(each - 12, each + 12, 80)
    sizes[-1] += 80 * each - sizes.sum()
    assert k.grouped_matmul_form(80, 80 * each, 250, 4096) == form
    for gather, out, acc in ((True, "f32", False), (False, "bf16", False), (True, "f32", True)):
        _check_wide(W, V, list(sizes), 4, gather, out, acc)


@pytest.mark.parametrize("sizes", [[1], [0, 7, 1], [16, 3, 0, 12, 17]])
@pytest.mark.parametrize("N,K", [(1, 4096), (200, 4096), (385, 7168)])
def test_matmul_few_tiles_in_parts(N, K, sizes):
    W, V = _wide(len(sizes), N, K)
    for gather, out, acc in ((True, "f32", False), (False, "bf16", False), (True, "f32", True)):
        _check_wide(W, V, sizes, 1, gather, out, acc)


def test_matmul_whole_numbers_are_exact():
    """Codes and scales that keep every sum below 2^24: equal to the integer product."""
    sizes, kk, N, K = [70, 1, 0, 190, 33], 3, 300, 1024
    g, ids = _plan(sizes, kk, 4)
    rng = np.random.default_rng(8)
    packed = rng.integers(0, 256, (len(sizes), N, K // 2), dtype=np.uint8)
    scales = np.full((len(sizes), N, K // 32), 128, np.uint8)  # codes times two: whole numbers up to 12
    W = k.MxExperts.from_matrices(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda())
    V = np.stack([mx.values(mx.unpack(p), s) for p, s in zip(packed, scales)])
    x = rng.integers(-15, 16, (ids.shape[0], K)).astype(np.float32)  # e4m3 holds these at any scale used
    a = k.Mx8Rows(*x.shape)
    k.mx8_quantize(a, torch.from_numpy(x).cuda())
    C = torch.empty(ids.size, N, device="cuda")
    k.grouped_matmul(C, a, W, g, gather=True)
    off, src = _sources(ids, len(sizes), True)
    assert np.array_equal(C[:off[-1]].double().cpu().numpy(), _want(off, src, x.astype(np.float64), V)[0])


def test_matmul_bad_values_stay_in_their_rows():
    sizes, kk, N, K = [20, 3, 50], 2, 140, 256
    g, ids = _plan(sizes, kk)
    W, V = _weights(3, N, K, 1)
    x = torch.randn(ids.shape[0], K, generator=torch.Generator().manual_seed(1))
    a = k.Mx8Rows(*x.shape)
    k.mx8_quantize(a, x.cuda())
    good = torch.empty(ids.size, N, device="cuda")
    k.grouped_matmul(good, a, W, g, gather=True)
    x[5, 200], x[9, 0] = float("inf"), float("nan")
    k.mx8_quantize(a, x.cuda())
    C = torch.empty(ids.size, N, device="cuda")
    k.grouped_matmul(C, a, W, g, gather=True)
    off, src = _sources(ids, 3, True)
    bad = torch.from_numpy(np.isin(src, (5, 9))).cuda()
    kept = off[-1]
    assert bool(torch.isnan(C[:kept][bad]).all()) and torch.equal(C[:kept][~bad], good[:kept][~bad])


def test_matmul_of_filled_operands_and_blobs():
    """Matrices quantised by the operand call (both orientations: the output and its
    input gradient), and the planes of equally spaced expert blobs."""
    E, d, f, kk = 3, 256, 384, 2
    gen = torch.Generator().manual_seed(6)
    w = torch.randn(E, f, d, generator=gen)
    g, ids = _plan([40, 0, 23], kk)
    fwd, bwd = k.MxExperts(E, f, d), k.MxExperts(E, d, f)
    for e in range(E):
        k.mx_quantize_operand(w[e].cuda(), fwd.operand(e), bwd.operand(e))
    for W, m in ((fwd, w.numpy()), (bwd, w.transpose(1, 2).contiguous().numpy())):
        V = np.stack([mx.values(*mx.quantize(v)) for v in m])
        a, A = _rows(ids.size, W.in_, 2)
        C = torch.empty(ids.size, W.rows, device="cuda")
        k.grouped_matmul(C, a, W, g)
        off, src = _sources(ids, E, False)
        want, mag = _want(off, src, A, V)
        assert (np.abs(C[:off[E]].double().cpu().numpy() - want) <= mag * (W.in_ / 32 + 11) * 2.0 ** -22).all()
    n = k.expert_bytes(d, f)
    blobs = torch.from_numpy(np.random.default_rng(3).integers(0, 256, (E, n), dtype=np.uint8)).cuda()
    at = f * d // 2
    blobs[:, at:at + f * d // 32] = 125
    gate, gs = blobs[:, :at].view(E, f, d // 2), blobs[:, at:at + f * d // 32].unflatten(1, (f, d // 32))
    W = k.MxExperts.from_matrices(gate, gs)
    assert W.struct.codes_stride == n
    a, A = _rows(ids.shape[0], d, 5)
    C = torch.empty(ids.size, f, device="cuda")
    k.grouped_matmul(C, a, W, g, gather=True)
    V = np.stack([mx.values(mx.unpack(p), s) for p, s in zip(gate.cpu().numpy(), gs.cpu().numpy())])
    off, src = _sources(ids, E, True)
    want, mag = _want(off, src, A, V)
    assert (np.abs(C[:off[E]].double().cpu().numpy() - want) <= mag * (d / 32 + 11) * 2.0 ** -22).all()


# ------------------------------------------------------------ weight gradients

def _wgrad_want(off, src, DY, X):
    w = np.stack([DY[off[e]:off[e + 1]].T @ X[src[off[e]:off[e + 1]]] for e in range(off.size - 1)])
    m = np.stack([np.abs(DY[off[e]:off[e + 1]]).T @ np.abs(X[src[off[e]:off[e + 1]]]) for e in range(off.size - 1)])
    return w, m


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("N,K,kk,pad", [(8, 8, 1, 0), (128, 256, 2, 8), (200, 328, 3, 0), (264, 520, 4, 16)])
def test_wgrad(N, K, kk, pad, sizes, gather, out):
    sizes = SIZES[sizes]
    ids = _ids(sizes, kk, 3) if sum(sizes) else np.full((4, kk), -1, np.int32)
    E, slots = len(sizes), ids.size
    g = k.ExpertGroups(E, kk, ids.shape[0])
    g.plan(torch.from_numpy(ids).cuda())
    gen = torch.Generator().manual_seed(N + K)
    dy = torch.randn(slots, N + pad, generator=gen).bfloat16().cuda()[:, :N]
    x = torch.randn(ids.shape[0] if gather else slots, K + pad, generator=gen).bfloat16().cuda()[:, :K]
    off, src = _sources(ids, E, gather)
    kept = off[E]
    dy[kept:] = float("nan")  # rows behind the groups take no part
    DY, X = dy.double().cpu().numpy(), x.double().cpu().numpy()
    want, mag = _wgrad_want(off, src, DY, X)
    dw = torch.full((E, N, K), 7.0, dtype=DT[out], device="cuda")
    k.grouped_wgrad(dw, dy, x, g, gather=gather)
    # an fp32 step (16 rows each) loses 2^-22 of the sum of magnitudes
    n = (off[1:] - off[:-1])[:, None, None]
    tol = mag * (n / 16 + 10) * 2.0 ** -22 + np.abs(want) * HALF[out]
    assert (np.abs(dw.double().cpu().numpy() - want) <= tol).all()
    again = torch.empty_like(dw)
    k.grouped_wgrad(again, dy, x, g, gather=gather)
    assert torch.equal(again, dw)
    if out == "f32":
        k.grouped_wgrad(dw, dy, x, g, gather=gather, accumulate=True)
        assert torch.equal(dw, again + again)
    assert k.device_error() == 0


# more tiles than two waves of single CTAs: pairs; groups of few rows and of many (in group
# order they keep four and six stages), columns that leave the odd CTA little or nothing
MANY = {"short": [200, 128, 129, 1, 0, 257], "long": [900, 400, 0, 513, 64, 463]}


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K,sizes", [(1032, 2056, "short"), (1032, 2056, "long"), (136, 264, "experts"), (72, 520, "experts")])
def test_wgrad_pairs(N, K, sizes, gather, out):
    kk = 2
    sizes = [int(n) for n in np.random.default_rng(N).integers(0, 70, 128)] if sizes == "experts" else MANY[sizes]
    g, ids = _plan(sizes, kk, 9)
    E, slots = len(sizes), ids.size
    off, src = _sources(ids, E, gather)
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    dy = torch.randn(slots, N + 8, generator=gen, device="cuda").bfloat16()[:, :N]
    x = torch.randn(ids.shape[0] if gather else slots, K, generator=gen, device="cuda").bfloat16()
    dy[off[E]:] = float("nan")
    dw = torch.full((E, N, K), 7.0, dtype=DT[out], device="cuda")
    k.grouped_wgrad(dw, dy, x, g, gather=gather)
    rows = torch.from_numpy(np.ascontiguousarray(src)).cuda().long()
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        DY, X = dy[s].double(), x[rows[s]].double()
        want, mag = DY.t() @ X, DY.abs().t() @ X.abs()
        tol = mag * ((off[e + 1] - off[e]) / 16 + 10) * 2.0 ** -22 + want.abs() * HALF[out]
        assert bool(((dw[e].double() - want).abs() <= tol).all()), e
    again = torch.empty_like(dw)
    k.grouped_wgrad(again, dy, x, g, gather=gather)
    assert torch.equal(again, dw)
    if out == "f32":
        k.grouped_wgrad(dw, dy, x, g, gather=gather, accumulate=True)
        assert torch.equal(dw, again + again)
    assert k.device_error() == 0


def test_wgrad_bad_values_stay_in_their_expert():
    sizes, kk, N, K = [30, 64, 5], 1, 136, 264
    g, ids = _plan(sizes, kk)
    gen = torch.Generator().manual_seed(1)
    dy, x = torch.randn(ids.size, N, generator=gen).bfloat16().cuda(), torch.randn(ids.size, K, generator=gen).bfloat16().cuda()
    good = torch.empty(3, N, K, device="cuda")
    k.grouped_wgrad(good, dy, x, g)
    dy[30, 3], x[30, 7] = float("nan"), float("inf")  # the first row of the second group
    dw = torch.empty_like(good)
    k.grouped_wgrad(dw, dy, x, g)
    assert torch.equal(dw[0], good[0]) and torch.equal(dw[2], good[2])
    assert bool(torch.isnan(dw[1, 3]).all()) and not bool(torch.isfinite(dw[1, :, 7]).any())


def test_wgrad_whole_numbers_are_exact():
    sizes, kk, N, K = [257, 3, 0, 64], 2, 72, 520
    g, ids = _plan(sizes, kk)
    rng = np.random.default_rng(2)
    dy, x = rng.integers(-20, 21, (ids.size, N)), rng.integers(-20, 21, (ids.shape[0], K))
    dw = torch.empty(len(sizes), N, K, device="cuda")
    t = lambda v: torch.from_numpy(v.astype(np.float32)).bfloat16().cuda()  # noqa: E731
    k.grouped_wgrad(dw, t(dy), t(x), g, gather=True)
    off, src = _sources(ids, len(sizes), True)
    assert np.array_equal(dw.double().cpu().numpy(), _wgrad_want(off, src, dy.astype(float), x.astype(float))[0])


def test_wgrad_against_differences():
    """d/dW of sum <dY_i, W_e x_i>: linear, so one difference gives it."""
    sizes, kk, N, K = [9, 0, 20], 2, 16, 24
    g, ids = _plan(sizes, kk)
    gen = torch.Generator().manual_seed(1)
    dy, x = torch.randn(ids.size, N, generator=gen).bfloat16().cuda(), torch.randn(ids.shape[0], K, generator=gen).bfloat16().cuda()
    dw = torch.empty(3, N, K, device="cuda")
    k.grouped_wgrad(dw, dy, x, g, gather=True)
    off, src = _sources(ids, 3, True)
    DY, X, rng = dy.double().cpu().numpy(), x.double().cpu().numpy(), np.random.default_rng(0)

    def f(W):
        return sum((DY[i] * (W[e] @ X[src[i]])).sum() for e in range(3) for i in range(off[e], off[e + 1]))
    for _ in range(3):
        v = rng.standard_normal(dw.shape)
        num = (f(v) - f(-v)) / 2
        assert abs((dw.double().cpu().numpy() * v).sum() - num) <= 2.0 ** -18 * np.abs(dw.double().cpu().numpy() * v).sum()


def test_capture_and_other_stream():
    """Plan, product and gradient in a graph that is replayed on new ids, and on a
    stream of their own."""
    E, kk, T, N, K = 6, 2, 90, 136, 256
    rng = np.random.default_rng(1)
    ids = [torch.from_numpy(rng.integers(-1, E, (T, kk)).astype(np.int32)).cuda() for _ in range(2)]
    W, _ = _weights(E, N, K, 1)
    gen = torch.Generator().manual_seed(1)
    x, dy = torch.randn(T, K, generator=gen).bfloat16().cuda(), torch.randn(T * kk, N, generator=gen).bfloat16().cuda()

    def state():
        return dict(g=k.ExpertGroups(E, kk, T), a=k.Mx8Rows(T, K), C=torch.zeros(T * kk, N, device="cuda"),
                    dw=torch.zeros(E, N, K, device="cuda"))

    def run(s, i):
        s["g"].plan(i)
        k.mx8_quantize(s["a"], x)
        s["C"].zero_()
        k.grouped_matmul(s["C"], s["a"], W, s["g"], gather=True)
        k.grouped_wgrad(s["dw"], dy, x, s["g"], gather=True)
    want = [state(), state()]
    for s, i in zip(want, ids):
        run(s, i)
    side, b = torch.cuda.Stream(), state()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(b, ids[0])
    torch.cuda.synchronize()
    assert torch.equal(b["C"], want[0]["C"]) and torch.equal(b["dw"], want[0]["dw"])
    c, now = state(), ids[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, now)
    for s, i in zip(want, ids):
        now.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c["C"], s["C"]) and torch.equal(c["dw"], s["dw"])
