"""The norm, the 8-bit rows and the grouped calls in the order of a stream: what they
write is complete before a kernel that loads weights early, and they start early
themselves only up to their own wait."""
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k
from test_gpu_weight_order import D, F, FULL, PROGRAMMATIC, READERS, _state, edges

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def state():
    t = _state()
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    t.update(norm=k.RmsNorm(D, 1e-6), rows=b(F, D), r=b(F, D), gain=torch.ones(D, device="cuda"), rstd=torch.ones(F, device="cuda"),
             dgain=torch.empty(D, device="cuda"), r8=k.Mx8Rows(F, D), G=k.ExpertGroups(4, 1, F),
             ids=torch.zeros(F, 1, dtype=torch.int32, device="cuda"), W=k.MxExperts(4, 64, D), C=b(F, 64), dW=b(4, 64, D),
             dy=b(F, 64))
    t["W"].codes.zero_(), t["W"].atoms.zero_()
    t["packed4"] = torch.zeros(4, 64, D // 2, dtype=torch.uint8, device="cuda")
    t["scales4"] = torch.zeros(4, 64, D // 32, dtype=torch.uint8, device="cuda")
    t["G"].plan(t["ids"])
    k.mx8_quantize(t["r8"], t["rows"])
    return t


WRITERS = {
    "norm_forward": lambda t, s: t["norm"].forward(t["plane"], t["rows"], t["wb"], t["r"], stream=s),
    "norm_backward": lambda t, s: t["norm"].backward(t["plane"], t["dgain"], t["rows"], t["rows"], t["rstd"], t["gain"], stream=s),
    "mx8_quantize": lambda t, s: k.mx8_quantize(t["r8"], t["rows"], stream=s),
    "mx8_dequantize": lambda t, s: k.mx8_dequantize(t["plane"], t["r8"], stream=s),
    "plan": lambda t, s: t["G"].plan(t["ids"], stream=s),
    "from_matrices": lambda t, s: k.MxExperts.from_matrices(t["packed4"], t["scales4"], stream=s),
    "grouped_matmul": lambda t, s: k.grouped_matmul(t["C"], t["r8"], t["W"], t["G"], stream=s),
    "grouped_wgrad": lambda t, s: k.grouped_wgrad(t["dW"], t["dy"], t["rows"], t["G"], stream=s),
    "combine": lambda t, s: k.combine(t["plane"], t["rows"], t["G"], stream=s),
    "combine_backward": lambda t, s: k.combine_backward(t["plane"], None, t["rows"], None, t["G"], stream=s),
}


@pytest.mark.parametrize("reader", READERS)
@pytest.mark.parametrize("writer", WRITERS)
def test_full_edge_behind_a_writer(state, writer, reader):
    one = len(edges(lambda s: (READERS[reader](state, s), READERS[reader](state, s)))) // 2 + 1  # kernels of a read
    kernels = len(edges(lambda s: [WRITERS[writer](state, s) for _ in range(2)])) // 2 + 1       # and of a write
    got = edges(lambda s: (WRITERS[writer](state, s), READERS[reader](state, s)))
    assert len(got) == one + kernels - 1 and got[kernels - 1] == FULL


@pytest.mark.parametrize("writer", WRITERS)
def test_they_wait_themselves(state, writer):
    assert set(edges(lambda s: [WRITERS[writer](state, s) for _ in range(3)])) == {PROGRAMMATIC}


def test_runs_behind_each_other_without_waiting_on_the_host():
    """Plan, rows, product and combine on new ids back to back, each result as that of the
    calls one at a time."""
    T, kk, E, N, K = 500, 2, 7, 384, 512
    gen = torch.Generator(device="cuda").manual_seed(3)
    w8 = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sc = torch.randint(120, 131, (E, N, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    W, G, a8 = k.MxExperts.from_matrices(w8, sc), k.ExpertGroups(E, kk, T), k.Mx8Rows(T, K)
    C = torch.empty(T * kk, N, device="cuda")
    batches = [(torch.randint(0, E, (T, kk), generator=gen, device="cuda", dtype=torch.int32),
                torch.randn(T, K, generator=gen, device="cuda")) for _ in range(12)]

    def run(ids, x, wait):
        out = torch.empty(T, N, device="cuda")
        for call in (lambda: G.plan(ids), lambda: k.mx8_quantize(a8, x), lambda: k.grouped_matmul(C, a8, W, G, gather=True),
                     lambda: k.combine(out, C, G)):
            call()
            if wait:
                torch.cuda.synchronize()
        return out
    fast = [run(*b, False) for b in batches]
    torch.cuda.synchronize()
    assert all(torch.equal(f, run(*b, True)) for f, b in zip(fast, batches))
