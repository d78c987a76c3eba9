"""Matrices of more than 2^31 elements through the norm, the 8-bit rows and the calls
grouped by expert: the first, the middle and the last rows equal those of small calls."""
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
T, N = 66001, 32768  # 2.16e9 elements
ENDS = ((0, 3), (65400, 65800), (T - 3, T))


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _big(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("pad", [0, 1])
def test_norm_and_rows_in_8_bits(pad):
    n = N - 8 * pad - pad  # with a pad rows are not aligned
    x, d, dy = (_big(T, n + pad, i)[:, :n] for i in range(3))
    norm, y, r, dx = k.RmsNorm(n, 1e-6), torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rstd, y8 = torch.empty(T, device="cuda"), k.Mx8Rows(T, n)
    norm.forward(y, x, d, r, rstd, None, y8)
    norm.backward(dx, None, dy, r, rstd, None, dy)
    codes, scales = y8.codes.view(T, -1), y8.scales.view(T, -1)
    v = torch.empty_like(x)
    k.mx8_dequantize(v, y8)
    q8 = k.Mx8Rows(T, n)
    k.mx8_quantize(q8, x)
    for a, b in ENDS:
        o = [torch.empty_like(x[a:b]) for _ in range(4)]
        s, s8, t8 = torch.empty(b - a, device="cuda"), k.Mx8Rows(b - a, n), k.Mx8Rows(b - a, n)
        norm.forward(o[0], x[a:b], d[a:b], o[1], s, None, s8)
        norm.backward(o[2], None, dy[a:b], o[1], s, None, dy[a:b])
        k.mx8_dequantize(o[3], s8)
        k.mx8_quantize(t8, x[a:b])
        for p, q in ((y, o[0]), (r, o[1]), (dx, o[2]), (rstd, s), (v, o[3]), (codes, s8.codes.view(b - a, -1)),
                     (scales, s8.scales.view(b - a, -1)), (q8.codes.view(T, -1), t8.codes.view(b - a, -1)),
                     (q8.scales.view(T, -1), t8.scales.view(b - a, -1))):
            assert torch.equal(p[a:b], q), a


def _plan(E, kk, tokens, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, E, (tokens, kk), generator=g, device="cuda", dtype=torch.int32)
    G = k.ExpertGroups(E, kk, tokens)
    G.plan(ids)
    return G, ids


def test_combine():
    G, ids = _plan(4, 2, T // 2 + 1, 1)
    slots, tokens = G.slots, G.tokens
    y, dout, w = _big(slots, N, 1), _big(tokens, N, 2), torch.rand(tokens, 2, device="cuda")
    out, dy, dw = torch.empty(tokens, N, device="cuda", dtype=torch.bfloat16), torch.empty_like(y), torch.empty_like(w)
    k.combine(out, y, G, w)
    k.combine_backward(dy, dw, dout, y, G, w)
    pos = G.pos.view(tokens, 2).long()
    for a, b in ((0, 5), (tokens // 2, tokens // 2 + 200), (tokens - 4, tokens)):
        want = sum(w[a:b, j, None] * y[pos[a:b, j]].float() for j in range(2))
        assert bool(((out[a:b].float() - want).abs() <= want.abs() * 2.0 ** -8 + 1e-6).all())
        for j in range(2):
            rows = pos[a:b, j]
            assert torch.equal(dy[rows], (w[a:b, j, None] * dout[a:b].float()).bfloat16())
            # products of two values up to 6, N of them; the kernel's sums are shorter
            dot = (y[rows].double() * dout[a:b].double()).sum(1)
            assert bool(((dw[a:b, j].double() - dot).abs() <= N * 36 * 2.0 ** -24).all())


@pytest.mark.parametrize("pair,E,rows,K", [(True, 4, T, 1024), (False, 1024, T // 8, 128)])
def test_result(pair, E, rows, K):
    """A result of more than 2^31 elements, of both kernels."""
    n = (1 << 31) // rows // 2 * 2 + 2
    G, ids = _plan(E, 1, rows, 2)
    gen = torch.Generator(device="cuda").manual_seed(4)
    assert (k.grouped_matmul_form(E, rows, n, K) == 256) == pair
    packed = torch.randint(0, 256, (E, n, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(120, 131, (E, n, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    W = k.MxExperts.from_matrices(packed, scales)
    x = torch.randn(rows, K, generator=gen, device="cuda")
    a8 = k.Mx8Rows(rows, K)
    k.mx8_quantize(a8, x)
    C = torch.empty(rows, n, device="cuda", dtype=torch.bfloat16)
    k.grouped_matmul(C, a8, W, G, gather=True)
    off, order = G.offsets.tolist(), G.order.long()
    for e in (0, E // 2, E - 1):  # the same group alone, rows in group order
        lo, hi = off[e], min(off[e + 1], off[e] + 300)
        if hi == lo:
            continue
        g1 = k.ExpertGroups(1, 1, hi - lo)
        g1.plan(torch.zeros(hi - lo, 1, dtype=torch.int32, device="cuda"))
        b8, c = k.Mx8Rows(hi - lo, K), torch.empty(hi - lo, n, device="cuda", dtype=torch.bfloat16)
        k.mx8_quantize(b8, x[order[lo:hi]])
        k.grouped_matmul(c, b8, k.MxExperts.from_matrices(packed[e:e + 1], scales[e:e + 1]), g1)
        # forms add in another order: the same to a rounding of bf16 and fp32 sums of K terms
        v = torch.empty(hi - lo, K, device="cuda")
        k.mx8_dequantize(v, b8)
        slack = v.abs().sum(1, keepdim=True) * 6 * 2.0 ** 3 * K / 32 * 2.0 ** -22
        assert bool(((C[lo:hi].float() - c.float()).abs() <= c.float().abs() * 2.0 ** -7 + slack).all()), e
    assert k.device_error() == 0


def test_rows_of_more_than_2_31_bytes():
    rows, K, n, E = 66000, 32768, 256, 3
    G, ids = _plan(E, 1, rows, 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    packed = torch.randint(0, 256, (E, n, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.full((E, n, K // 32), 122, device="cuda", dtype=torch.uint8)
    W = k.MxExperts.from_matrices(packed, scales)
    x = _big(rows, K, 5)
    a8, C = k.Mx8Rows(rows, K), torch.empty(rows, n, device="cuda")
    k.mx8_quantize(a8, x)
    k.grouped_matmul(C, a8, W, G, gather=True)
    in_order = x[G.order.long()]
    k.mx8_quantize(a8, in_order)
    D = torch.empty_like(C)
    k.grouped_matmul(D, a8, W, G)
    assert torch.equal(C, D) and k.device_error() == 0


def test_wgrad():
    E, n, K, tokens = 20, 10240, 10752, 640  # 2.2e9 gradients
    G, ids = _plan(E, 1, tokens, 6)
    dy, x = _big(tokens, n, 1), _big(tokens, K, 2)
    dw = torch.empty(E, n, K, device="cuda", dtype=torch.bfloat16)
    k.grouped_wgrad(dw, dy, x, G, gather=True)
    off, order = G.offsets.tolist(), G.order.long()
    for e in (0, 10, E - 1):
        lo, hi = off[e], off[e + 1]
        for r in (slice(0, 64), slice(n - 64, n)):
            a, b = dy[lo:hi, r].double(), x[order[lo:hi]].double()
            want, mag = a.t() @ b, a.abs().t() @ b.abs()
            tol = mag * ((hi - lo) / 16 + 10) * 2.0 ** -22 + want.abs() * 2.0 ** -8
            assert bool(((dw[e, r].double() - want).abs() <= tol).all()), e
    assert k.device_error() == 0
