"""Matrices of more than 2^31 elements, and rows of a result that far apart: the
last rows equal those of small calls."""
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
T, F = 66001, 32800  # 2.16e9 elements; more rows than one SwiGLU or dequantisation launch takes
ENDS = ((0, 3), (65400, 65800), (T - 3, T))


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _big(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("pad", [0, 1])
def test_swiglu(pad):
    g, u, dh = (_big(T, F + pad, i)[:, :F] for i in range(3))
    ck, h = k.SwigluCheckpoint(T, F), torch.empty_like(g)
    k.swiglu_forward(h, ck, g, u)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    k.swiglu_backward(dg, du, dh, ck)
    for a, b in ENDS:
        c, want = k.SwigluCheckpoint(b - a, F), [torch.empty_like(g[a:b]) for _ in range(3)]
        k.swiglu_forward(want[0], c, g[a:b], u[a:b])
        k.swiglu_backward(want[1], want[2], dh[a:b], c)
        for x, y in zip((h, dg, du), want):
            assert torch.equal(x[a:b], y), a


@pytest.mark.parametrize("pad", [0, 1])
def test_quantise_and_values(pad):
    x = _big(T, F + pad, 3)[:, :F]
    row, col = k.MxOperand(T, F), k.MxOperand(F, T)
    k.mx_quantize_operand(x, row, col)
    y = torch.empty(T, F + pad, device="cuda", dtype=torch.bfloat16)[:, :F]
    k.mx_dequantize(y, row)
    codes = row.codes.view(T, -1)
    for a, b in ENDS:
        op, want = k.MxOperand(b - a, F), torch.empty_like(y[a:b])
        k.mx_quantize_operand(x[a:b], op)
        k.mx_dequantize(want, op)
        assert torch.equal(codes[a:b], op.codes.view(b - a, -1)) and torch.equal(y[a:b], want), a
    # columns, by a transposed copy
    yt = torch.empty(F, T + pad, device="cuda", dtype=torch.bfloat16)[:, :T]
    k.mx_dequantize(yt, col)
    for a, b in ((0, 70), (F - 70, F)):
        op, want = k.MxOperand(b - a, T), torch.empty(b - a, T, device="cuda", dtype=torch.bfloat16)
        k.mx_quantize_operand(x[:, a:b].t().contiguous(), op)
        k.mx_dequantize(want, op)
        assert torch.equal(yt[a:b], want), a


# forms: pairs with TMA stores and without, single CTAs, split
@pytest.mark.parametrize("M,N,K,ld", [(3001, 3336, 3300, 1 << 20), (3001, 3333, 3300, (1 << 20) + 1), (3041, 2, 10900, 1 << 20),
                                      (1388, 4558, 300, 1 << 21), (9, 3000, 3001, 1 << 28), (7, 3001, 700, (1 << 29) + 1)])
def test_product_rows_far_apart(M, N, K, ld):
    A, B = k.MxOperand(M, K), k.MxOperand(N, K)
    k.mx_quantize_operand(_big(M, K, 4), A)
    k.mx_quantize_operand(_big(N, K, 5), B)
    want = torch.empty(M, N, device="cuda")
    k.mx_matmul(want, A, B)
    C = torch.empty(M, ld, device="cuda")[:, :N]
    k.mx_matmul(C, A, B)
    assert torch.equal(C, want)
    k.mx_matmul(C, A, B, accumulate=True)
    assert torch.equal(C, 2 * want)
    assert k.device_error() == 0


@pytest.mark.parametrize("E", [896, 897])
def test_balance(E):
    n, kk = 2400001, 4
    l = _big(n, E, 6)
    ids = torch.randint(0, E, (n, kk), device="cuda", dtype=torch.int32)
    bal = k.BalanceLoss(E, kk, 0.1)
    loss, counts, valid = torch.empty(1, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda"), \
        torch.empty(1, dtype=torch.int32, device="cuda")
    bal.forward(loss, counts, valid, l, ids)
    assert int(valid) == n and torch.equal(counts.long(), torch.bincount(ids.view(-1).long(), minlength=E))
    # random logits and choices: p and f are even up to their sampling
    assert abs(float(loss) / 0.1 - 1) < 1e-3
    dl, d = torch.empty_like(l), torch.full((1,), 1e9, device="cuda")
    bal.backward(dl, l, ids, counts, valid, d)
    for a, b in ((0, 5), (2396700, 2397000), (n - 5, n)):
        want = torch.empty_like(l[a:b])
        bal.backward(want, l[a:b], ids[a:b], counts, valid, d)
        assert torch.equal(dl[a:b], want) and bool(want.any()), a
