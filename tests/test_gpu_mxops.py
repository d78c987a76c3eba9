"""MXFP4 operands on the GPU: quantisation along rows and columns code for code
against the oracle's conversion, the values they stand for, and the product
against the fp64 product of those values, over sizes from 1, odd sizes, strides,
both types, and the forms (tiles, split along K) the product takes."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _x(rows, cols, dt, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    return x.to(dt).cuda()[:, :cols]


def _np(x):
    return x.detach().float().cpu().numpy()


def _check_operand(op, x):
    """Codes and atoms of `op` against the oracle's conversion of x (numpy)."""
    codes, scales = ref.quantize(x)
    rows, n = x.shape
    got = ref.unpack(op.codes.cpu().numpy().reshape(rows, -1))
    s, clean = ref.atoms_to_scales(op.atoms.cpu().numpy(), rows, n)
    assert np.array_equal(s, scales)
    assert np.array_equal(got, codes)
    assert clean, "bytes past the matrix"
    return codes, scales


def _filled(rows, n):
    """An operand whose buffers hold 0xff, so that what a call leaves shows."""
    op = k.MxOperand(rows, n)
    op.codes.fill_(255)
    op.atoms.fill_(255)
    return op


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 31, 0), (1, 7168, 0), (33, 32, 0), (128, 256, 8), (129, 257, 3),
                                           (300, 100, 4), (31, 1000, 1), (1000, 127, 0), (512, 640, 0), (70, 33, 7), (300, 391, 9)])
def test_quantize_both_ways(rows, cols, pad, dt):
    x = _x(rows, cols, DT[dt], rows * 1000 + cols, pad)
    row, col = _filled(rows, cols), _filled(cols, rows)
    k.mx_quantize_operand(x, row, col)
    only_row, only_col = _filled(rows, cols), _filled(cols, rows)
    k.mx_quantize_operand(x, only_row)
    k.mx_quantize_operand(x, None, only_col)
    torch.cuda.synchronize()
    _check_operand(row, _np(x))
    _check_operand(col, _np(x).T)
    for a, b in ((row, only_row), (col, only_col)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.atoms, b.atoms)


def _edge_matrix():
    """32 x 64: rounding midpoints at several exponents, zeros, -0, subnormals,
    the largest values, a maximum just below a power of two."""
    rng = np.random.default_rng(5)
    m = np.zeros((32, 64), np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for r, ex in enumerate((-130, -100, -20, -1, 0, 1, 5, 60, 120)):
        m[r] = np.tile(np.concatenate([mids, -mids]), 4) * 2.0 ** ex
        m[r, ::32] = 6.0 * 2.0 ** ex
    m[10] = -0.0
    m[11] = 1e-40 * np.arange(64)
    m[12] = np.linspace(-3.4e38, 3.4e38, 64)
    m[13] = rng.standard_normal(64) * 3
    m[13, 5] = m[13, 40] = 7.9999995
    return m


@pytest.mark.parametrize("along", ["row", "col"])
def test_quantize_edges(along):
    m = _edge_matrix()
    x = torch.from_numpy(m if along == "row" else np.ascontiguousarray(m.T)).cuda()
    op = _filled(32, 64)
    k.mx_quantize_operand(x, op, None) if along == "row" else k.mx_quantize_operand(x, None, op)
    torch.cuda.synchronize()
    codes, scales = _check_operand(op, m)
    y = torch.empty(32, 64, device="cuda")
    k.mx_dequantize(y, op)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), ref.values(codes, scales))


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_nonfinite_block_reads_back_as_nan_and_spreads_to_its_products(bad):
    x = _np(_x(40, 96, torch.float32, 3)).copy()
    x[7, 40] = bad
    xd = torch.from_numpy(x).cuda()
    row, col, w = k.MxOperand(40, 96), k.MxOperand(96, 40), k.MxOperand(50, 96)
    k.mx_quantize_operand(xd, row, col)
    k.mx_quantize_operand(_x(50, 96, torch.float32, 4), w)
    y, yt, C = torch.empty(40, 96, device="cuda"), torch.empty(96, 40, device="cuda"), torch.empty(40, 50, device="cuda")
    k.mx_dequantize(y, row)
    k.mx_dequantize(yt, col)
    k.mx_matmul(C, row, w)
    nan, nan_t = np.isnan(y.cpu().numpy()), np.isnan(yt.cpu().numpy())
    want = np.zeros((40, 96), bool)
    want[7, 32:64] = True
    assert np.array_equal(nan, want)
    want_t = np.zeros((96, 40), bool)
    want_t[40, :32] = True
    assert np.array_equal(nan_t, want_t)
    c = np.isnan(C.cpu().numpy())
    assert c[7].all() and c.sum() == 50


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,pad", [(1, 1, 0), (3, 33, 0), (130, 300, 5), (256, 512, 8), (40, 300, 4),
                                        (133, 1000, 0), (70, 49, 7), (9, 47, 9), (5, 290, 6)])
def test_dequantize(rows, n, pad, dt):
    op = k.MxOperand(rows, n)
    k.mx_quantize_operand(_x(rows, n, torch.float32, 11), op)
    y = torch.full((rows, n + pad), 77.0, dtype=DT[dt], device="cuda")
    k.mx_dequantize(y[:, :n], op)
    codes, scales = ref.quantize(_np(_x(rows, n, torch.float32, 11)))
    assert np.array_equal(_np(y[:, :n]).astype(np.float64), ref.values(codes, scales)[:, :n])
    assert bool((y[:, n:] == 77).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dequantize_many_units_per_thread(dt):
    """A matrix of more units than the grid has threads, against its row blocks."""
    rows, n = 4100, 5216
    x = _x(rows, n, torch.float32, 12)
    op = k.MxOperand(rows, n)
    k.mx_quantize_operand(x, op)
    y = torch.empty(rows, n, dtype=DT[dt], device="cuda")
    k.mx_dequantize(y, op)
    for r in range(0, rows, 1000):
        part = x[r:r + 1000]
        op, want = k.MxOperand(part.shape[0], n), torch.empty_like(y[r:r + 1000])
        k.mx_quantize_operand(part, op)
        k.mx_dequantize(want, op)
        assert torch.equal(y[r:r + 1000], want)


def _bound(a, b, out):
    """Element bound of the product: each fp32 step (at most K / 64 + a final
    sum over 8 ranks, and the alignment of the 64 products of a step) loses at
    most 2^-22 of the largest running magnitude, itself at most sum |a||b|; then
    half a step of the output type."""
    mag = np.abs(a) @ np.abs(b).T
    steps = a.shape[1] / 64 + 10
    half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    return mag * steps * 2.0 ** -22 + np.abs(a @ b.T) * half


def _operands(M, N, K, seed):
    A, B = k.MxOperand(M, K), k.MxOperand(N, K)
    xa, xb = _x(M, K, torch.float32, seed), _x(N, K, torch.float32, seed + 1)
    k.mx_quantize_operand(xa, A)
    k.mx_quantize_operand(xb, B)
    va, vb = (ref.values(*ref.quantize(_np(x)))[:, :K] for x in (xa, xb))
    return A, B, va, vb


SIZES = [(1, 1, 1), (1, 128, 256), (1, 200, 32), (2, 129, 31), (5, 1000, 700), (16, 7168, 1536), (17, 300, 4096),
         (33, 128, 7168), (64, 1536, 7168), (65, 40, 520), (100, 1, 300), (128, 256, 257), (129, 255, 1024),
         (200, 1537, 96), (256, 384, 2048), (333, 1000, 1112), (1, 20000, 64), (40, 20001, 256)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K, out):
    A, B, va, vb = _operands(M, N, K, 7 * M + N + K)
    C = torch.full((M, N + 3), 5.0, dtype=DT[out], device="cuda")
    k.mx_matmul(C[:, :N], A, B)
    torch.cuda.synchronize()
    assert k.device_error() == 0
    want = va @ vb.T
    err = np.abs(_np(C[:, :N]).astype(np.float64) - want)
    assert (err <= _bound(va, vb, out)).all(), float((err / np.maximum(_bound(va, vb, out), 1e-300)).max())
    assert bool((C[:, N:] == 5).all()), "columns past N"


@pytest.mark.parametrize("M,N,K", [(4096, 1536, 512), (1500, 7168, 300), (2049, 5000, 256), (700, 24000, 128)])
def test_matmul_many_tiles(M, N, K):
    """More tiles than SMs: 128- and 256-column tiles, ragged at both ends."""
    A, B, va, vb = _operands(M, N, K, M + N)
    C = torch.empty(M, N, device="cuda")
    k.mx_matmul(C, A, B)
    torch.cuda.synchronize()
    assert k.device_error() == 0
    a, b = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda()
    mag = a.abs() @ b.abs().t()
    tol = mag * (K / 64 + 10) * 2.0 ** -22 + (a @ b.t()).abs() * 2.0 ** -24
    assert bool(((C.double() - a @ b.t()).abs() <= tol).all())


@pytest.mark.parametrize("M,N,K", [(3, 500, 2048), (300, 256, 640), (4096, 1600, 256)])
def test_matmul_accumulates_and_repeats(M, N, K):
    A, B, va, vb = _operands(M, N, K, 99)
    C0 = _x(M, N, torch.float32, 8)
    C, D = C0.clone(), C0.clone()
    k.mx_matmul(C, A, B, accumulate=True)
    for _ in range(3):
        D.copy_(C0)
        k.mx_matmul(D, A, B, accumulate=True)
        assert torch.equal(C, D)
    want = _np(C0).astype(np.float64) + va @ vb.T
    # the addition to C rounds once more
    tol = _bound(va, vb, "f32") + np.abs(want) * 2.0 ** -24
    assert (np.abs(_np(C) - want) <= tol).all()


@pytest.mark.parametrize("rows,n", [(1, 32), (130, 96), (200, 1024)])
def test_stored_matrix(rows, n):
    """An expert's plane pair as an operand: scale byte 255 drops its group."""
    rng = np.random.default_rng(rows)
    packed = rng.integers(0, 256, (rows, n // 2), dtype=np.uint8)
    scales = rng.integers(118, 134, (rows, n // 32), dtype=np.uint8)
    scales[rows // 2, 0] = 255
    scales[0, -1] = 0
    op = k.MxOperand.from_matrix(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), rows, n)
    A, _, va, _ = _operands(9, 1, n, 4)
    C = torch.empty(9, rows, device="cuda")
    k.mx_matmul(C, A, op)
    v = ref.values(ref.unpack(packed), np.where(scales == 255, 0, scales).astype(np.uint8))
    s, clean = ref.atoms_to_scales(op.atoms.cpu().numpy(), rows, n)
    assert clean and np.array_equal(s, np.where(scales == 255, 0, scales))
    dropped = ref.values(ref.unpack(packed), scales)
    dropped[np.isnan(dropped)] = 0.0
    assert (np.abs(_np(C) - va @ dropped.T) <= _bound(va, v, "f32") + 1e-30).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 40, 70), (50, 33, 129), (257, 130, 300)])
def test_linear_gradients(T, N, K, dt):
    """Output, input gradient and weight gradient of a linear layer in MXFP4:
    each against the formula on the quantised values, and the input gradient
    against differences of <dy, y> (the product is linear in a row's values)."""
    x, w, dy = _x(T, K, DT[dt], 1), _x(N, K, DT[dt], 2), _x(T, N, DT[dt], 3)
    o = dict(xr=(T, K), xc=(K, T), wr=(N, K), wc=(K, N), gr=(T, N), gc=(N, T))
    o = {n: k.MxOperand(*s) for n, s in o.items()}
    k.mx_quantize_operand(x, o["xr"], o["xc"])
    k.mx_quantize_operand(w, o["wr"], o["wc"])
    k.mx_quantize_operand(dy, o["gr"], o["gc"])
    y, dx, dw = (torch.empty(s, device="cuda") for s in ((T, N), (T, K), (N, K)))
    k.mx_matmul(y, o["xr"], o["wr"])
    k.mx_matmul(dx, o["gr"], o["wc"])
    k.mx_matmul(dw, o["gc"], o["xc"])

    def q(v):
        return ref.values(*ref.quantize(v))[:, :v.shape[1]]
    X, W, G = _np(x), _np(w), _np(dy)
    for got, a, b in ((y, q(X), q(W)), (dx, q(G), q(W.T)), (dw, q(G.T), q(X.T))):
        assert (np.abs(_np(got) - a @ b.T) <= _bound(a, b, "f32")).all()
    # differences: f(x) = <q(dy), x q(W^T)^T>, one entry of x moved by h either way
    rng = np.random.default_rng(0)
    Xd = X.astype(np.float64)

    def f(v):
        return float((q(G) * (v @ q(W.T))).sum())
    for _ in range(5):
        i, j = rng.integers(T), rng.integers(K)
        h = 2.0 ** -3
        e = np.zeros_like(Xd)
        e[i, j] = h
        diff = (f(Xd + e) - f(Xd - e)) / (2 * h)
        slack = 1e-9 * float(np.abs(q(G)) .sum() * np.abs(Xd).max() * np.abs(q(W.T)).max())
        assert abs(float(dx[i, j]) - diff) <= _bound(q(G), q(W.T), "f32")[i, j] + slack


def test_other_stream_and_graph():
    """The calls run on the stream that is current, and replay from a graph with
    new inputs."""
    M, N, K = 70, 260, 1100
    x, w = _x(M, K, torch.float32, 21), _x(N, K, torch.float32, 22)
    A, B, C = k.MxOperand(M, K), k.MxOperand(N, K), torch.empty(M, N, device="cuda")

    def step():
        k.mx_quantize_operand(x, A)
        k.mx_quantize_operand(w, B)
        k.mx_matmul(C, A, B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    first = C.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    C.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, first)
    x.mul_(-2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, -2.0 * first)
    assert k.device_error() == 0


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(2048, 1537, 160, 0), (1100, 3333, 512, 3), (4096, 1000, 288, 8), (3000, 2064, 64, 0),
                                       (257, 12000, 1056, 1), (2500, 1300, 1, 4), (4096, 1537, 2100, 0),
                                       (2300, 3333, 1500, 3), (1500, 7001, 900, 8), (2500, 7168, 260, 0),
                                       (9000, 5000, 96, 0), (3001, 4600, 1056, 2),
                                       (2304, 2901, 2500, 3), (2200, 2950, 4000, 2), (4095, 1536, 7168, 8),
                                       (2100, 5400, 10000, 0)])
def test_matmul_pairs(M, N, K, pad, out):
    """Products large enough for CTA pairs: rows of C aligned for wide stores or
    not, ragged row and column tiles of every width, a K of one block and less."""
    A, B, va, vb = _operands(M, N, K, M + 3 * N)
    C = torch.full((M, N + pad), 5.0, dtype=DT[out], device="cuda")
    k.mx_matmul(C[:, :N], A, B)
    a, b = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda()
    want = a @ b.t()
    tol = (a.abs() @ b.abs().t()) * (K / 64 + 10) * 2.0 ** -22 + want.abs() * (2.0 ** -8 if out == "bf16" else 2.0 ** -24)
    assert bool(((C[:, :N].double() - want).abs() <= tol).all())
    assert bool((C[:, N:] == 5).all())
    if out == "f32":
        k.mx_matmul(C[:, :N], A, B, accumulate=True)
        tol = tol * 2 + 2 * want.abs() * 2.0 ** -24
        assert bool(((C[:, :N].double() - 2 * want).abs() <= tol).all())
        assert bool((C[:, N:] == 5).all())
    torch.cuda.synchronize()
    assert k.device_error() == 0


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(129, 1536, 7168, 0), (160, 1001, 7000, 3), (192, 1536, 5000, 4), (255, 1400, 7168, 0),
                                       (333, 1500, 8200, 1), (160, 128, 4000, 0), (300, 37, 9000, 2), (1000, 130, 9000, 0)])
def test_matmul_split_beyond_one_row_tile(M, N, K, pad, out):
    """A long K split over CTAs, several tiles of 64 and 128 rows of A."""
    A, B, va, vb = _operands(M, N, K, M + N)
    C = torch.full((M, N + pad), 5.0, dtype=DT[out], device="cuda")
    k.mx_matmul(C[:, :N], A, B)
    want = va @ vb.T
    tol = _bound(va, vb, out)
    assert bool((np.abs(_np(C[:, :N]).astype(np.float64) - want) <= tol).all())
    assert bool((C[:, N:] == 5).all())
    again = torch.empty_like(C)
    k.mx_matmul(again[:, :N], A, B)
    assert torch.equal(again[:, :N], C[:, :N])
    if out == "f32":
        k.mx_matmul(C[:, :N], A, B, accumulate=True)
        assert bool((np.abs(_np(C[:, :N]).astype(np.float64) - 2 * want) <= 2 * tol + np.abs(want) * 2.0 ** -23).all())
    assert k.device_error() == 0


def test_matmul_nan_stays_in_its_rows_and_columns():
    """Non-finite blocks in a CTA-pair product reach their own row and column only
    (tiles reach past the matrices, and the tail of K past the blocks)."""
    M, N, K = 2050, 5000, 2000
    x, w = _x(M, K, torch.float32, 1), _x(N, K, torch.float32, 2)
    x[700, 40] = float("nan")
    w[4999, 1999] = float("inf")
    A, B, C = k.MxOperand(M, K), k.MxOperand(N, K), torch.empty(M, N, device="cuda")
    k.mx_quantize_operand(x, A)
    k.mx_quantize_operand(w, B)
    k.mx_matmul(C, A, B)
    bad = torch.isnan(C)
    assert bool(bad[700].all()) and bool(bad[:, 4999].all()) and int(bad.sum()) == M + N - 1


def test_weights_written_by_a_call_are_seen_by_the_next():
    """Calls that load weights before their predecessor on the stream has finished
    see what a dequantisation, a product or a quantisation wrote just before."""
    d, f = 1024, 512
    gen = torch.Generator(device="cuda").manual_seed(3)
    blob = torch.empty(k.shared_expert_bytes(d, f) // 2, dtype=torch.bfloat16, device="cuda")
    view = [k.shared_expert_view(blob.data_ptr(), d, f)]
    x, ws = torch.randn(1, d, generator=gen, device="cuda"), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    got, want = torch.empty(1, d, device="cuda"), torch.empty(1, d, device="cuda")
    ops = [k.MxOperand(f, d), k.MxOperand(f, d), k.MxOperand(d, f)]
    planes = [blob[:f * d].view(f, d), blob[f * d:2 * f * d].view(f, d), blob[2 * f * d:].view(d, f)]
    ident = k.MxOperand(f, f)
    k.mx_quantize_operand(torch.eye(f, device="cuda"), ident)
    down_t = k.MxOperand(d, f)
    for it in range(20):
        ws_ = [torch.randn(o.rows, o.in_, generator=gen, device="cuda") * 0.05 for o in ops]
        for o, w in zip(ops, ws_):
            k.mx_quantize_operand(w, o)
        k.mx_quantize_operand(ws_[2], down_t)
        torch.cuda.synchronize()
        # the last plane by a dequantisation, or by a product with the identity
        order = (2, 1, 0) if it % 2 else (0, 1, 2)
        for i in order:
            if it % 4 == 2 and i == 2:
                k.mx_matmul(planes[2], down_t, ident)
            else:
                k.mx_dequantize(planes[i], ops[i])
        k.shared_forward(got, x, 1, view, d, f, ws)
        torch.cuda.synchronize()
        k.shared_forward(want, x, 1, view, d, f, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    # an expert's packed gate plane written by the quantiser, then its GEMV
    packed, scales = torch.empty(f, d // 2, dtype=torch.uint8, device="cuda"), torch.full((f, d // 32), 124, device="cuda",
                                                                                          dtype=torch.uint8)
    y, y2 = torch.empty(f, device="cuda"), torch.empty(f, device="cuda")
    op = k.MxOperand(f, d, codes=packed.view(-1))
    for _ in range(20):
        w = torch.randn(f, d, generator=gen, device="cuda")
        torch.cuda.synchronize()
        k.mx_quantize_operand(w, op)
        k.matmul_mxfp4(y, x, packed, scales, f, d)
        torch.cuda.synchronize()
        k.matmul_mxfp4(y2, x, packed, scales, f, d)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
