"""Every form that the MXFP4 product takes, by name: single CTAs with 16, 32, 64 and
128 columns, whole and split over 2, 4 and 8 CTAs, and CTA pairs with 192, 256 and
384, each at ragged sizes, in both types, with rows of C that TMA stores take and
rows that it does not, accumulating, with several tiles per CTA, with non-finite
blocks, and repeated.  The form is asserted, so that a change of the choice shows
here instead of leaving a form untested."""
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BOTH = ("f32", "bf16")

# form (pair, columns, ranks), output types, M, N, K
CASES = [
    ((False, 16, 1), BOTH, 7, 3001, 700), ((False, 16, 1), BOTH, 3, 20001, 200),
    ((False, 16, 2), BOTH, 7, 6914, 6739), ((False, 16, 4), BOTH, 9, 3000, 3001), ((False, 16, 4), BOTH, 2, 2873, 2858),
    ((False, 16, 8), BOTH, 1, 1536, 7168), ((False, 16, 8), BOTH, 16, 1001, 5000),
    ((False, 32, 1), BOTH, 17, 3001, 1300), ((False, 32, 1), BOTH, 27, 20001, 300),
    ((False, 32, 2), BOTH, 31, 5888, 7656), ((False, 32, 4), BOTH, 22, 2433, 5332), ((False, 32, 8), BOTH, 20, 1537, 7168),
    ((False, 64, 1), BOTH, 333, 1000, 1112), ((False, 64, 1), BOTH, 917, 3423, 70), ((False, 64, 1), BOTH, 129, 20001, 300),
    ((False, 64, 2), BOTH, 3041, 2, 10900), ((False, 64, 4), BOTH, 523, 304, 7683), ((False, 64, 8), BOTH, 64, 1537, 7168),
    ((False, 64, 8), BOTH, 1000, 37, 7000),
    ((False, 128, 1), BOTH, 928, 1321, 145), ((False, 128, 1), BOTH, 1388, 4558, 300),
    ((True, 192, 1), BOTH, 1536, 1538, 3000), ((True, 192, 1), BOTH, 3912, 609, 1824), ((True, 192, 1), BOTH, 3001, 3333, 3300),
    ((True, 192, 1), BOTH, 6863, 2530, 200),
    ((True, 256, 1), BOTH, 2132, 1635, 6483), ((True, 256, 1), BOTH, 1563, 4486, 3196),
    ((True, 256, 1), ("bf16",), 2306, 7168, 1500), ((True, 256, 1), BOTH, 2510, 6600, 4000),
    ((True, 384, 1), BOTH, 1753, 3124, 3295), ((True, 384, 1), BOTH, 3520, 5664, 3161), ((True, 384, 1), BOTH, 1304, 8422, 9000),
]
FLAT = [(form, dt, M, N, K) for form, dts, M, N, K in CASES for dt in dts]


def _operand(rows, n, seed):
    """An operand and the values it stands for, in fp64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, n, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda").float())
    op, v = k.MxOperand(rows, n), torch.empty(rows, n, device="cuda")
    k.mx_quantize_operand(x, op)
    k.mx_dequantize(v, op)
    return op, v.double()


def _on_this_device(form, dt, M, N, K):
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("sizes chosen for 152 SMs")
    assert k.mx_matmul_form(M, N, K, DT[dt]) == form


@pytest.mark.parametrize("form,dt,M,N,K", FLAT)
def test_form(form, dt, M, N, K):
    _on_this_device(form, dt, M, N, K)
    (A, a), (B, b) = _operand(M, K, 1), _operand(N, K, 2)
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    # each fp32 step (K / 64, and the join of up to 8 ranks) loses at most 2^-22 of the
    # largest running magnitude; half a step of the output type
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    tol = mag * (K / 64 + 10) * 2.0 ** -22 + want.abs() * half
    # rows of C one element past a 16-byte unit, and rows of whole units
    for pad in (3, -N % 8 + 8, 0):
        C = torch.full((M, N + pad), 5.0, dtype=DT[dt], device="cuda")
        k.mx_matmul(C[:, :N], A, B)
        assert bool(((C[:, :N].double() - want).abs() <= tol).all()), pad
        assert bool((C[:, N:] == 5).all())
        again = torch.zeros_like(C)
        k.mx_matmul(again[:, :N], A, B)
        assert torch.equal(again[:, :N], C[:, :N])
        if dt == "f32":
            k.mx_matmul(C[:, :N], A, B, accumulate=True)
            assert bool(((C[:, :N].double() - 2 * want).abs() <= 2 * tol + want.abs() * 2.0 ** -23).all()), pad
            assert bool((C[:, N:] == 5).all())
    assert k.device_error() == 0


# N a multiple of 8: the rows of C are whole 16-byte units, and pairs store by TMA
@pytest.mark.parametrize("form,dt,M,N,K", [((True, 192, 1), "f32", 3001, 3336, 3300), ((True, 192, 1), "bf16", 3001, 3336, 3300),
                                           ((True, 256, 1), "f32", 2510, 6600, 4000), ((True, 256, 1), "bf16", 2306, 7168, 1500),
                                           ((True, 256, 1), "f32", 4096, 7168, 4096), ((True, 256, 1), "bf16", 4096, 7168, 1536),
                                           ((True, 384, 1), "f32", 3520, 5664, 3161), ((True, 384, 1), "bf16", 4096, 1536, 7168)])
def test_pairs_by_tma(form, dt, M, N, K):
    """Against the same values with rows of C that TMA does not take."""
    _on_this_device(form, dt, M, N, K)
    (A, _), (B, _) = _operand(M, K, 3), _operand(N, K, 4)
    C, D = (torch.full((M, N + p), 5.0, dtype=DT[dt], device="cuda") for p in (8, 1))
    k.mx_matmul(C[:, :N], A, B)
    k.mx_matmul(D[:, :N], A, B)
    assert torch.equal(C[:, :N], D[:, :N]) and bool((C[:, N:] == 5).all()) and bool((D[:, N:] == 5).all())
    if dt == "f32":
        k.mx_matmul(C[:, :N], A, B, accumulate=True)
        assert torch.equal(C[:, :N], 2 * D[:, :N]) and bool((C[:, N:] == 5).all())
    assert k.device_error() == 0


@pytest.mark.parametrize("form,dt,M,N,K", [(f, "f32", m, n, kk) for f, _, m, n, kk in CASES
                                           if (m, n) in ((9, 3000), (22, 2433), (333, 1000), (523, 304), (1388, 4558), (3001, 3333),
                                                         (1563, 4486), (3520, 5664))])
def test_nonfinite_blocks_stay_in_their_rows_and_columns(form, dt, M, N, K):
    """Tiles reach past the matrices, and the last k-step past the blocks."""
    _on_this_device(form, dt, M, N, K)
    x, w = torch.randn(M, K, device="cuda"), torch.randn(N, K, device="cuda")
    x[M // 3, 40] = float("nan")
    w[N - 1, K - 1] = float("inf")
    A, B, C = k.MxOperand(M, K), k.MxOperand(N, K), torch.empty(M, N, device="cuda")
    k.mx_quantize_operand(x, A)
    k.mx_quantize_operand(w, B)
    k.mx_matmul(C, A, B)
    bad = torch.isnan(C)
    assert bool(bad[M // 3].all()) and bool(bad[:, N - 1].all()) and int(bad.sum()) == M + N - 1
    assert k.device_error() == 0
