"""Argument refusals of the norm, the 8-bit rows and the calls grouped by expert (no
GPU: each is refused before any CUDA call), their host arithmetic, and the binding's
checks of devices, types and shapes."""
import ctypes

import pytest

from mxfp4_routed_expert_select_gb300 import k3moe as k

torch = pytest.importorskip("torch")
EINVAL = k.K3MOE_EINVAL
P, Q, R, S = 4096, 2 << 20, 4 << 20, 6 << 20  # pointers that are never followed


def addr(ref):
    """Address behind a byref (0 for None)."""
    return 0 if ref is None else ctypes.cast(ref, ctypes.c_void_p).value


def pack(S, *a):
    return S.pack(*(0 if v is None else v for v in a))


def rows8(rows=4, n=64, codes=P, scales=P):
    return ctypes.byref(k.Mx8RowsStruct(codes, scales, rows, n))


def groups(E=3, kk=2, T=5, offsets=P, order=P, pos=P, ws=P, nws=1 << 40):
    return ctypes.byref(k.GroupsStruct(offsets, order, pos, ws, nws, E, kk, T))


def experts(E=3, rows=40, n=128, codes=P, atoms=P, cs=40 * 64, as_=2048):
    return ctypes.byref(k.MxExpertsStruct(codes, atoms, cs, as_, E, rows, n))


def test_sizes():
    L = k.lib()
    assert L.k3moe_mx8_codes_bytes(3, 33) == 3 * 64 and L.k3moe_mx8_scales_bytes(3, 33) == 12
    assert L.k3moe_mx8_codes_bytes(1 << 30, 1 << 20) == 1 << 50 and L.k3moe_mx8_scales_bytes(2, 129) == 16
    for f in (L.k3moe_mx8_codes_bytes, L.k3moe_mx8_scales_bytes):
        assert f(0, 1) == f(1, 0) == f(1, (1 << 20) + 1) == f((1 << 30) + 1, 1) == -1
    assert L.k3moe_norm_workspace(0) == L.k3moe_norm_workspace(32769) == 0 and L.k3moe_norm_workspace(7168) >= 7168 * 4
    assert L.k3moe_groups_workspace(0, 1) == L.k3moe_groups_workspace(1025, 1) == L.k3moe_groups_workspace(5, 0) == 0
    assert L.k3moe_groups_workspace(5, (1 << 30) + 1) == 0
    assert L.k3moe_groups_workspace(1024, 1 << 30) > L.k3moe_groups_workspace(1024, 1) > 0


BAD_ROWS = (None, rows8(0), rows8(4, 0), rows8(codes=None), rows8(codes=P + 8), rows8(scales=None), rows8(scales=P + 4),
            rows8(n=(1 << 20) + 1))


def test_rows_in_8_bits():
    for f in (lambda o, x, dt, ld: k.lib().k3moe_mx8_quantize(o, x, dt, ld, None),
              lambda o, x, dt, ld: k.lib().k3moe_mx8_dequantize(x, dt, ld, o, None)):
        for bad in BAD_ROWS:
            assert f(bad, P, 0, 1 << 20) == EINVAL
        for x, dt, ld in ((None, 0, 64), (P + 2, 0, 64), (P + 1, 1, 64), (P, 2, 64), (P, 0, 63), (P, 0, (1 << 40) + 1)):
            assert f(rows8(), x, dt, ld) == EINVAL


def test_norm_forward():
    good = dict(y=Q, ldy=64, r=R, ldr=64, rstd=P, y8=None, x=P, ldx=64, d=S, ldd=64, gain=P, dt=0, T=4, n=64, eps=1e-6)
    for bad in (dict(x=None), dict(x=P + 2), dict(ldx=63), dict(d=None), dict(ldd=63), dict(d=S + 1), dict(y=None),
                dict(ldy=0), dict(y=Q + 2), dict(ldr=63), dict(r=R + 3), dict(y=R), dict(rstd=P + 2), dict(gain=P + 1),
                dict(dt=2), dict(dt=-1), dict(T=0), dict(T=(1 << 30) + 1), dict(n=0), dict(n=32769, ldx=1 << 20),
                dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(y8=rows8(5)), dict(y8=rows8(4, 63)),
                dict(y=P, ldy=72), dict(y=S, ldy=72), dict(r=P, ldr=72), dict(r=S, ldr=72), *(dict(y8=b) for b in BAD_ROWS[1:])):
        a = {**good, **bad}
        d = pack(k.NORM_FORWARD, a["y"], a["ldy"], a["r"], a["ldr"], a["rstd"], addr(a["y8"]), a["x"], a["ldx"], a["d"],
                 a["ldd"], a["gain"], a["dt"], a["T"], a["n"], a["eps"])
        assert k.lib().k3moe_norm_forward(d, None) == EINVAL, bad
    assert k.lib().k3moe_norm_forward(None, None) == EINVAL


def test_norm_backward():
    ws = k.lib().k3moe_norm_workspace(64)
    good = dict(dx=Q, lddx=64, dg=P, dy=R, lddy=64, dr=S, lddr=64, r=P, ldr=64, rstd=P, gain=P, dt=0, T=4, n=64, ws=P, nws=ws)
    for bad in (dict(dx=None), dict(dx=Q + 2), dict(lddx=63), dict(dy=None), dict(lddy=63), dict(dr=S + 2), dict(lddr=63),
                dict(r=None), dict(ldr=63), dict(rstd=None), dict(rstd=P + 2), dict(gain=None), dict(gain=P + 2),
                dict(dg=P + 2), dict(ws=None), dict(ws=P + 8), dict(nws=ws - 1), dict(dt=3), dict(T=0), dict(n=0),
                dict(dx=R, lddx=72), dict(dx=S, lddx=72), dict(dx=P, lddx=72)):
        a = {**good, **bad}
        d = pack(k.NORM_BACKWARD, a["dx"], a["lddx"], a["dg"], a["dy"], a["lddy"], a["dr"], a["lddr"], a["r"], a["ldr"],
                 a["rstd"], a["gain"], a["ws"], a["nws"], a["dt"], a["T"], a["n"], 0)
        assert k.lib().k3moe_norm_backward(d, None) == EINVAL, bad
    assert k.lib().k3moe_norm_backward(None, None) == EINVAL


BAD_GROUPS = (None, groups(0), groups(1025), groups(kk=0), groups(kk=33), groups(T=0), groups(T=1 << 30), groups(offsets=None),
              groups(order=None), groups(pos=None), groups(offsets=P + 2), groups(order=P + 2), groups(pos=P + 1), groups(ws=None), groups(ws=P + 8), groups(nws=1000),
              groups(T=10000, nws=k.lib().k3moe_groups_workspace(3, 20000) - 1))


def test_plan():
    L = k.lib()
    for bad in BAD_GROUPS:
        assert L.k3moe_groups_plan(bad, P, None) == EINVAL
    for ids in (None, P + 2):
        assert L.k3moe_groups_plan(groups(), ids, None) == EINVAL


def test_matmul():
    good = dict(C=P, dt=0, ldc=40, A=rows8(10, 128), W=experts(), g=groups(), gather=0, acc=0)
    bad = [dict(C=None), dict(C=P + 2), dict(dt=4), dict(ldc=39), dict(dt=1, acc=1), dict(A=rows8(9, 128)),
           dict(A=rows8(4, 128), gather=1), dict(A=rows8(10, 256)), dict(W=None), dict(W=experts(E=4)), dict(W=experts(n=96)),
           dict(W=experts(n=64), A=rows8(10, 64)), dict(W=experts(codes=P + 16)), dict(W=experts(codes=None)),
           dict(W=experts(atoms=P + 8)), dict(W=experts(atoms=None)), dict(W=experts(rows=0)), dict(W=experts(cs=40 * 64 - 32)),
           dict(W=experts(cs=40 * 64 + 16)), dict(W=experts(as_=512)), dict(W=experts(as_=2056)), dict(W=experts(cs=1 << 40)),
           dict(W=experts(rows=1 << 14, cs=1 << 20, as_=1 << 20), g=groups(T=1 << 23), A=rows8(1 << 24, 128), ldc=1 << 14),
           *(dict(A=b) for b in BAD_ROWS), *(dict(g=b) for b in BAD_GROUPS)]
    for b in bad:
        a = {**good, **b}
        d = pack(k.GROUPED_MATMUL, a["C"], a["ldc"], addr(a["A"]), addr(a["W"]), addr(a["g"]), a["dt"], a["gather"], a["acc"])
        assert k.lib().k3moe_grouped_matmul(d, None) == EINVAL, b
    assert k.lib().k3moe_grouped_matmul(None, None) == EINVAL


def test_stored_experts():
    L = k.lib()
    for W, sc, st in ((None, P, 160), (experts(), None, 160), (experts(), P, 159), (experts(), P, (1 << 40) + 1),
                      (experts(n=96), P, 160), (experts(codes=P + 16), P, 160), (experts(as_=512), P, 160),
                      (experts(E=0), P, 160), (experts(E=1025), P, 160)):
        assert L.k3moe_mx_experts_from_matrices(W, sc, st, None) == EINVAL


def test_form_query():
    L, o = k.lib(), ctypes.byref(ctypes.c_int32())
    assert L.k3moe_grouped_matmul_form(1, 1, 1, 128, o) == k.K3MOE_OK
    for a in ((0, 1, 1, 128), (1025, 1, 1, 128), (1, 0, 1, 128), (1, (1 << 30) + 1, 1, 128), (1, 1, 0, 128), (1, 1, 1, 0),
              (1, 1, 1, 64), (1, 1, 1, 192)):
        assert L.k3moe_grouped_matmul_form(*a, o) == EINVAL
    assert L.k3moe_grouped_matmul_form(1, 1, 1, 128, None) == EINVAL
    for E, slots, N, n in ((1, 1, 1, 128), (1024, 1 << 30, 1 << 20, 1 << 20), (8, 1000, 7168, 1536)):
        assert k.grouped_matmul_form(E, slots, N, n) in (16, 32, 64, 256)


def test_wgrad():
    good = dict(dw=P, dt=0, dy=P, lddy=16, x=P, ldx=24, xr=10, N=16, K=24, g=groups(), gather=0, acc=0)
    bad = [dict(dw=None), dict(dw=P + 8), dict(dt=2), dict(dt=1, acc=1), dict(dy=None), dict(dy=P + 8), dict(lddy=8),
           dict(lddy=20), dict(x=None), dict(x=P + 2), dict(ldx=16), dict(ldx=28), dict(xr=9), dict(xr=4, gather=1), dict(N=12),
           dict(N=0), dict(K=20), dict(K=0), dict(xr=(1 << 30) + 1),
           dict(N=1 << 18, K=1 << 19, lddy=1 << 18, ldx=1 << 19, g=groups(E=1000)), *(dict(g=b) for b in BAD_GROUPS)]
    for b in bad:
        a = {**good, **b}
        d = pack(k.GROUPED_WGRAD, a["dw"], a["dy"], a["lddy"], a["x"], a["ldx"], addr(a["g"]), a["dt"], a["xr"], a["N"], a["K"],
                 a["gather"], a["acc"])
        assert k.lib().k3moe_grouped_wgrad(d, None) == EINVAL, b
    assert k.lib().k3moe_grouped_wgrad(None, None) == EINVAL


def test_combine():
    good = dict(o=P, ldo=64, y=Q, ldy=64, dt=0, n=64, g=groups(), w=P)
    both = [dict(o=None), dict(o=P + 2), dict(ldo=63), dict(y=Q + 2), dict(ldy=63), dict(dt=2), dict(n=0), dict(w=P + 2),
            dict(n=(1 << 20) + 1, ldo=1 << 21, ldy=1 << 21), dict(g=groups(T=1 << 25), n=1 << 20, ldo=1 << 20, ldy=1 << 20),
            *(dict(g=b) for b in BAD_GROUPS)]
    for b in both + [dict(y=None), dict(o=Q)]:
        a = {**good, **b}
        d = pack(k.COMBINE, a["o"], a["ldo"], a["y"], a["ldy"], a["w"], addr(a["g"]), a["dt"], a["n"], 0)
        assert k.lib().k3moe_combine(d, None) == EINVAL, b
    good.update(dy=R, lddy=64, dw=P)
    for b in both + [dict(y=None), dict(dy=None), dict(dy=R + 2), dict(lddy=63), dict(dy=P), dict(w=None), dict(dw=P + 2),
                     dict(dy=Q, lddy=72)]:
        a = {**good, **b}
        d = pack(k.COMBINE_BACKWARD, a["dy"], a["lddy"], a["dw"], a["o"], a["ldo"], a["y"], a["ldy"], a["w"], addr(a["g"]),
                 a["dt"], a["n"])
        assert k.lib().k3moe_combine_backward(d, None) == EINVAL, b
    assert k.lib().k3moe_combine(None, None) == EINVAL and k.lib().k3moe_combine_backward(None, None) == EINVAL


def test_packed_descriptions_have_the_header_s_layout():
    """Sizes and the place of the last field, by the C compiler."""
    import shutil
    import subprocess
    import tempfile
    from conftest import ROOT
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    last = {"norm_forward": ("NORM_FORWARD", "eps"), "norm_backward": ("NORM_BACKWARD", "accumulate"),
            "grouped_matmul": ("GROUPED_MATMUL", "accumulate"), "grouped_wgrad": ("GROUPED_WGRAD", "accumulate"),
            "combine": ("COMBINE", "accumulate"), "combine_backward": ("COMBINE_BACKWARD", "n")}
    src = "#include <stdio.h>\n#include \"k3moe.h\"\nint main(void) {\n" + "".join(
        'printf("%%d %%d\\n", (int)sizeof(k3moe_%s_desc), (int)offsetof(k3moe_%s_desc, %s));\n' % (n, n, f)
        for n, (_, f) in last.items()) + "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        r = subprocess.run([gcc, "-I", ROOT + "/include", "-x", "c", "-", "-o", d + "/a"], input=src, text=True,
                           capture_output=True)
        assert r.returncode == 0, r.stderr
        out = subprocess.run([d + "/a"], capture_output=True, text=True).stdout.split()
    for i, (S, f) in enumerate(last.values()):
        S = getattr(k, S)
        marks = S.unpack(S.pack(*range(1, 1 + len(S.unpack(bytes(S.size))))))
        assert S.size == int(out[2 * i]), f
        data = bytearray(S.size)
        probe = S.pack(*([0] * (len(marks) - 1) + [1]))
        data[:] = probe
        first = next(j for j, v in enumerate(data) if v)
        assert first // 4 * 4 == int(out[2 * i + 1]), f


@pytest.fixture(params=["objects on the CPU too", "objects on GPU 0"])
def on(request):
    """Sets the GPU that an object says it is on."""
    def set_gpu(o):
        if request.param.endswith("0"):
            o.gpu = 0
        return o
    return set_gpu


def test_binding_refuses_tensors_elsewhere(on):
    x, f = torch.zeros(4, 128), torch.zeros(4)
    norm, r8, g = on(k.RmsNorm(128, 1e-6, device="cpu")), on(k.Mx8Rows(4, 128, device="cpu")), on(k.ExpertGroups(3, 2, 4, device="cpu"))
    W = on(k.MxExperts(3, 8, 128, device="cpu"))
    b = x.bfloat16()
    for call in (lambda: norm.forward(x.clone(), x), lambda: norm.forward(None, x, y8=r8),
                 lambda: norm.backward(x.clone(), None, x, x, f), lambda: k.mx8_quantize(r8, x), lambda: k.mx8_dequantize(x, r8),
                 lambda: g.plan(torch.zeros(4, 2, dtype=torch.int32)), lambda: k.grouped_matmul(torch.zeros(8, 8), r8, W, g),
                 lambda: k.grouped_wgrad(torch.zeros(3, 128, 128), b, b, g), lambda: k.combine(x, x, g),
                 lambda: k.combine_backward(x, None, x, None, g),
                 lambda: k.MxExperts.from_matrices(torch.zeros(3, 8, 64, dtype=torch.uint8), torch.zeros(3, 8, 4, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="GPU"):
            call()


class _OnGpu(torch.Tensor):
    """A CPU tensor that says it is on GPU 0: the checks behind the device's."""

    @staticmethod
    def of(t):
        return t.as_subclass(_OnGpu)

    def get_device(self):
        return 0


def test_binding_refuses_types_and_shapes():
    o = _OnGpu.of
    x, g = o(torch.zeros(4, 128)), k.ExpertGroups(3, 2, 4, device="cpu")
    norm, r8, W = k.RmsNorm(128, 1e-6, device="cpu"), k.Mx8Rows(4, 128, device="cpu"), k.MxExperts(3, 8, 128, device="cpu")
    for v in (norm, r8, g, W):
        v.gpu = 0
    h, f = o(torch.zeros(4, 128).bfloat16()), o(torch.zeros(4))
    for call, err in ((lambda: norm.forward(h, x), TypeError), (lambda: norm.forward(x, x, h), TypeError),
                      (lambda: norm.forward(x, o(torch.zeros(4, 64))), ValueError),
                      (lambda: norm.forward(x, x, rstd=o(torch.zeros(5))), ValueError),
                      (lambda: norm.forward(x, x, gain=o(torch.zeros(128).bfloat16())), ValueError),
                      (lambda: norm.backward(x, None, x, h, f), TypeError),
                      (lambda: k.mx8_quantize(r8, o(torch.zeros(5, 128))), ValueError),
                      (lambda: k.mx8_quantize(r8, o(torch.zeros(4, 128).half())), TypeError),
                      (lambda: g.plan(o(torch.zeros(4, 2, dtype=torch.int64))), ValueError),
                      (lambda: g.plan(o(torch.zeros(4, 3, dtype=torch.int32))), ValueError),
                      (lambda: g.plan(o(torch.zeros(5, 2, dtype=torch.int32))), ValueError),
                      (lambda: g.plan(o(torch.zeros(0, 2, dtype=torch.int32))), ValueError),
                      (lambda: k.grouped_matmul(o(torch.zeros(8, 9)), r8, W, g), ValueError),
                      (lambda: k.grouped_wgrad(o(torch.zeros(4, 8, 8)), h, h, g), ValueError),
                      (lambda: k.grouped_wgrad(o(torch.zeros(3, 8, 16).transpose(1, 2)), h, h, g), ValueError),
                      (lambda: k.grouped_wgrad(o(torch.zeros(3, 8, 8)), x, x, g), TypeError),
                      (lambda: k.combine(h, x, g), (TypeError, ValueError)),
                      (lambda: k.MxExperts(3, 8, 128, codes=o(torch.zeros(3, 8, 32, dtype=torch.uint8))), ValueError),
                      (lambda: k.MxExperts(3, 8, 96, device="cpu"), k.K3Error), (lambda: k.MxExperts(1025, 8, 128), k.K3Error),
                      (lambda: k.ExpertGroups(3, 33, 4, device="cpu"), k.K3Error), (lambda: k.RmsNorm(0, 1e-6, device="cpu"), k.K3Error),
                      (lambda: k.Mx8Rows(0, 5, device="cpu"), k.K3Error)):
        with pytest.raises(err):
            call()


def test_a_call_before_the_first_plan_is_refused():
    g, x = k.ExpertGroups(3, 2, 4, device="cpu"), _OnGpu.of(torch.zeros(0, 16))
    g.gpu = 0
    with pytest.raises(k.K3Error):
        k.combine(x, _OnGpu.of(torch.zeros(0, 16)), g, stream=0)
