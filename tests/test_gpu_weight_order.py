"""Kernels that load weights before their predecessor has completed are full
dependents of a call that may have written weights: seen in the edges of captured
graphs, where a programmatic dependency shows as such."""
import ctypes

import pytest
import torch

import synth
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
D, F = 1024, 512
FULL, PROGRAMMATIC = 0, 1


class Edge(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def edges(call):
    """Types of the edges of a chain of kernels that `call(stream)` enqueues, in order."""
    cu = ctypes.CDLL("libcuda.so.1")
    for _ in range(2):  # first-time set-up happens outside the capture
        call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h, g, n = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()
    assert cu.cuStreamBeginCapture_v2(h, 1) == 0  # this thread's calls only
    try:
        call(s)
    finally:
        assert cu.cuStreamEndCapture(h, ctypes.byref(g)) == 0
    try:
        assert cu.cuGraphGetEdges_v2(g, None, None, None, ctypes.byref(n)) == 0
        a, b, e = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (Edge * n.value)()
        assert cu.cuGraphGetEdges_v2(g, a, b, e, ctypes.byref(n)) == 0
        after = {x: (y, t.type) for x, y, t in zip(a, b, e)}
        assert len(after) == n.value, "a chain"
        at, out = (set(a) - set(b)).pop(), []
        while at in after:
            at, t = after[at]
            out.append(t)
        assert len(out) == n.value
        return out
    finally:
        cu.cuGraphDestroy(g)


def _state():
    g = torch.Generator(device="cuda").manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = dict(w=t(F, D), x=t(1, D), y=torch.empty(F, device="cuda"), out=torch.empty(1, D, device="cuda"),
              ws=torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))
    st["packed"] = torch.empty(F, D // 2, dtype=torch.uint8, device="cuda")
    st["scales"] = torch.full((F, D // 32), 124, dtype=torch.uint8, device="cuda")
    st["op"] = k.MxOperand(F, D, codes=st["packed"].view(-1))
    st["blob"] = torch.zeros(k.shared_expert_bytes(D, F) // 2, dtype=torch.bfloat16, device="cuda")
    st["plane"] = st["blob"][:F * D].view(F, D)
    st["shared"] = [k.shared_expert_view(st["blob"].data_ptr(), D, F)]
    st["eye"] = k.MxOperand(D, D)
    k.mx_quantize_operand(torch.eye(D, device="cuda"), st["eye"])
    k.mx_quantize_operand(st["w"], st["op"])
    st["ck"] = k.SwigluCheckpoint(F, D)
    st["wb"] = st["w"].bfloat16()
    st["expert_blob"] = torch.empty(k.expert_bytes(D, F), dtype=torch.uint8, device="cuda")
    keep = k.pack_expert(st["expert_blob"], synth.expert(3, 0, 0, D, F), D, F)
    torch.cuda.synchronize()
    st["expert"] = k.expert_view(st["expert_blob"].data_ptr(), D, F)
    st["gemv_ws"] = torch.empty(k.expert_gemv_workspace(D, F), dtype=torch.uint8, device="cuda")
    del keep
    return st


WRITERS = {
    "mx_quantize": lambda t, s: k.mx_quantize(t["packed"], t["scales"], t["w"], F, D, stream=s),
    "mx_quantize_operand": lambda t, s: k.mx_quantize_operand(t["w"], t["op"], stream=s),
    "mx_dequantize": lambda t, s: k.mx_dequantize(t["plane"], t["op"], stream=s),
    "mx_matmul": lambda t, s: k.mx_matmul(t["plane"], t["op"], t["eye"], stream=s),
    "swiglu_forward": lambda t, s: k.swiglu_forward(t["plane"], t["ck"], t["wb"], t["wb"], stream=s),
}
READERS = {
    "matmul_mxfp4": lambda t, s: k.matmul_mxfp4(t["y"], t["x"], t["packed"], t["scales"], F, D, stream=s),
    "shared_forward": lambda t, s: k.shared_forward(t["out"], t["x"], 1, t["shared"], D, F, t["ws"], stream=s),
    "expert_gemv": lambda t, s: k.expert_gemv(t["out"], t["x"], t["expert"], D, F, t["gemv_ws"], stream=s),
}


@pytest.mark.parametrize("reader", READERS)
@pytest.mark.parametrize("writer", WRITERS)
def test_full_edge_behind_a_writer(writer, reader):
    t = _state()
    one = len(edges(lambda s: (READERS[reader](t, s), READERS[reader](t, s)))) // 2 + 1  # kernels of a read
    got = edges(lambda s: (WRITERS[writer](t, s), READERS[reader](t, s)))
    assert len(got) == one and got[0] == FULL


@pytest.mark.parametrize("reader", READERS)
def test_programmatic_edges_elsewhere(reader):
    t = _state()
    assert set(edges(lambda s: [READERS[reader](t, s) for _ in range(3)])) == {PROGRAMMATIC}
    # the writers themselves touch nothing before their wait
    assert edges(lambda s: [WRITERS["mx_quantize_operand"](t, s) for _ in range(3)]) == [PROGRAMMATIC] * 2
    # a writer outside a capture does not reach into it
    WRITERS["mx_dequantize"](t, torch.cuda.current_stream())
    assert set(edges(lambda s: [READERS[reader](t, s) for _ in range(3)])) == {PROGRAMMATIC}


def test_the_batch_one_layer():
    """Its router rows are loaded early: behind a product that wrote them, not."""
    E, K = 32, 4
    blobs = torch.empty((E, k.expert_bytes(D, F)), dtype=torch.uint8, device="cuda")
    keep = [k.pack_expert(blobs[e], synth.expert(9, 0, e, D, F), D, F) for e in range(E)]
    torch.cuda.synchronize()
    Wr = torch.zeros(E, D, dtype=torch.bfloat16, device="cuda")
    op = k.MxOperand(E, D)
    k.mx_quantize_operand(torch.randn(E, D, device="cuda"), op)
    L = k.Layer(E, K, D, F, Wr.view(torch.int16), [k.expert_view(b.data_ptr(), D, F) for b in blobs], max_tokens=1)
    try:
        assert L.mx_t1()
        x, out = torch.randn(D, device="cuda"), torch.empty(D, device="cuda")
        run = lambda s: L.forward(x, 1, out, stream=s)  # noqa: E731
        assert edges(lambda s: (run(s), run(s))) == [PROGRAMMATIC]
        assert edges(lambda s: (k.mx_dequantize(Wr, op, stream=s), run(s)))[0] == FULL
        torch.cuda.synchronize()
        assert k.device_error() == 0
    finally:
        L.close()
    del keep


def test_eager_calls_follow_a_writer():
    """Weights written on the stream just before, by calls that last long enough for
    an early load to come too soon."""
    t = _state()
    T = torch.empty(8192, 8192, device="cuda")
    big = k.MxOperand(8192, 8192)
    k.mx_quantize_operand(torch.randn(8192, 8192, device="cuda"), big)
    want = torch.empty_like(t["y"])
    for i in range(20):
        w = torch.randn(F, D, device="cuda") * 2.0 ** (i % 5)
        torch.cuda.synchronize()
        k.mx_dequantize(T, big)
        k.mx_quantize_operand(w, t["op"])
        READERS["matmul_mxfp4"](t, None)
        torch.cuda.synchronize()
        k.matmul_mxfp4(want, t["x"], t["packed"], t["scales"], F, D)
        torch.cuda.synchronize()
        assert torch.equal(t["y"], want)
