"""Argument refusals of the operand, SwiGLU-checkpoint and balance-loss calls
(no GPU: each is refused before any CUDA call), and their host arithmetic."""
import ctypes

import pytest

from mxfp4_routed_expert_select_gb300 import k3moe as k

EINVAL = k.K3MOE_EINVAL
P = 4096  # a pointer that is never followed


def op(rows=8, n=64, codes=P, atoms=P):
    return ctypes.byref(k.MxOperandStruct(codes, atoms, rows, n))


def test_sizes():
    L = k.lib()
    assert L.k3moe_mx_operand_codes_bytes(1, 1) == 16
    assert L.k3moe_mx_operand_codes_bytes(3, 33) == 3 * 32
    assert L.k3moe_mx_operand_codes_bytes(1 << 30, 1 << 30) == (1 << 30) * (1 << 29)
    assert L.k3moe_mx_operand_atoms_bytes(1, 1) == 1024
    assert L.k3moe_mx_operand_atoms_bytes(129, 257) == 2 * 4 * 512
    for f in (L.k3moe_mx_operand_codes_bytes, L.k3moe_mx_operand_atoms_bytes, L.k3moe_swiglu_ckpt_bytes):
        assert f(0, 1) == -1 and f(1, 0) == -1 and f(-1, 5) == -1
    assert L.k3moe_mx_operand_codes_bytes(1, (1 << 30) + 1) == -1
    assert L.k3moe_swiglu_ckpt_bytes(2, 33) == 2 * 2 * (64 + 2)
    assert L.k3moe_swiglu_ckpt_bytes(1 << 20, 4096) == 2 * (1 << 20) * (4096 + 128)  # past 32 bits
    assert L.k3moe_balance_workspace(0) == 0 and L.k3moe_balance_workspace(1025) == 0
    assert L.k3moe_balance_workspace(1024) >= 12 * 1024


@pytest.mark.parametrize("row,col,x,dt,rows,cols,ld", [
    (None, None, P, 0, 8, 64, 64),                 # nothing to write
    (op(), None, None, 0, 8, 64, 64),
    (op(), None, P, 2, 8, 64, 64),                 # unknown type
    (op(), None, P, 0, 0, 64, 64),
    (op(), None, P, 0, 8, 64, 63),                 # short stride
    (op(), None, P + 2, 0, 8, 64, 64),             # fp32 off its element size
    (op(), None, P + 1, 1, 8, 64, 64),             # bf16 off its element size
    (op(9), None, P, 0, 8, 64, 64),                # operand of another shape
    (op(), op(8, 64), P, 0, 8, 64, 64),            # the column operand is cols x rows
    (op(codes=P + 8), None, P, 0, 8, 64, 64),
    (op(atoms=0), None, P, 0, 8, 64, 64),
])
def test_quantize_refusals(row, col, x, dt, rows, cols, ld):
    assert k.lib().k3moe_mx_quantize_operand(row, col, x, dt, rows, cols, ld, None) == EINVAL


def test_matrix_and_dequantize_refusals():
    L = k.lib()

    def mat(packed=P, scales=P, rows=8, n=64):
        return ctypes.byref(k.Mat(packed, scales, rows, n))
    for o, m in ((op(), None), (None, mat()), (op(), mat(packed=2 * P)), (op(), mat(rows=9)), (op(), mat(n=96)),
                 (op(n=60), mat(n=60)), (op(), mat(scales=P + 4)), (op(), mat(scales=None))):
        assert L.k3moe_mx_operand_from_matrix(o, m, None) == EINVAL
    for y, dt, ld, o in ((None, 0, 64, op()), (P, 5, 64, op()), (P, 0, 63, op()), (P, 0, 64, None), (P + 2, 0, 64, op()),
                         (P, 0, 64, op(rows=0))):
        assert L.k3moe_mx_dequantize(y, dt, ld, o, None) == EINVAL


@pytest.mark.parametrize("C,dt,ldc,A,B,acc", [
    (None, 0, 8, op(), op(), 0),
    (P, 3, 8, op(), op(), 0),
    (P, 0, 7, op(), op(), 0),
    (P + 1, 1, 8, op(), op(), 0),
    (P, 0, 8, op(), op(n=96), 0),                  # other reduction lengths
    (P, 0, 8, None, op(), 0),
    (P, 0, 8, op(), op(rows=-1), 0),
    (P, 1, 8, op(), op(), 1),                      # accumulation in bf16
    (P, 0, 8, op(atoms=P + 4), op(), 0),
])
def test_matmul_refusals(C, dt, ldc, A, B, acc):
    assert k.lib().k3moe_mx_matmul(C, dt, ldc, A, B, acc, None) == EINVAL


def test_swiglu_refusals():
    L = k.lib()
    T, f = 4, 40
    n = L.k3moe_swiglu_ckpt_bytes(T, f)
    good = dict(h=P, ldh=f, ck=P, n=n, g=P, ldg=f, u=P, ldu=f, dt=0, T=T, f=f)
    for bad in (dict(h=None), dict(ldh=f - 1), dict(ck=None), dict(ck=P + 8), dict(n=n - 1), dict(g=P + 2), dict(ldg=0),
                dict(u=None), dict(ldu=f - 1), dict(dt=7), dict(T=0), dict(f=0)):
        a = {**good, **bad}
        assert L.k3moe_swiglu_forward(a["h"], a["ldh"], a["ck"], a["n"], a["g"], a["ldg"], a["u"], a["ldu"], a["dt"],
                                      a["T"], a["f"], None) == EINVAL, bad
        b = dict(dg=a["g"], du=a["u"] and a["u"] + 64, dh=a["h"])
        assert L.k3moe_swiglu_backward(b["dg"], a["ldg"], b["du"], a["ldu"], b["dh"], a["ldh"], a["ck"], a["n"],
                                       a["dt"], a["T"], a["f"], None) == EINVAL, bad
    assert L.k3moe_swiglu_backward(P, f, P, f, P, f, P, n, 0, T, f, None) == EINVAL  # dg and du the same


def test_balance_refusals():
    L = k.lib()
    ws = L.k3moe_balance_workspace(32)
    good = dict(loss=P, counts=P, n=P, logits=P, dt=0, ld=32, ids=P, mask=None, T=4, E=32, k=2, rule=0, ws=P, nws=ws,
                dl=2 * P, ldd=32, dloss=P, w=P, dw=P)
    both = (dict(logits=None), dict(dt=9), dict(ld=31), dict(ids=None), dict(ids=P + 2), dict(T=0), dict(E=0),
            dict(E=1025, ld=1025, ldd=1025), dict(k=0), dict(k=33), dict(rule=3), dict(rule=-1), dict(counts=None),
            dict(n=None), dict(logits=P + 1))
    fwd = (dict(loss=None), dict(ws=None), dict(ws=P + 4), dict(nws=ws - 1), dict(loss=P + 2))
    bwd = (dict(dl=None), dict(ldd=31), dict(dloss=None), dict(w=None), dict(dw=None), dict(dl=P, ldd=64),
           dict(dw=P + 1))
    for bad in both + fwd:
        a = {**good, **bad}
        assert L.k3moe_balance_forward(a["loss"], a["counts"], a["n"], a["logits"], a["dt"], a["ld"], a["ids"],
                                       a["mask"], a["T"], a["E"], a["k"], 0.1, a["rule"], a["ws"], a["nws"],
                                       None) == EINVAL, bad
    for bad in both + bwd:
        a = {**good, **bad}
        assert L.k3moe_balance_backward(a["dl"], a["ldd"], a["logits"], a["dt"], a["ld"], a["ids"], a["mask"],
                                        a["counts"], a["n"], a["dloss"], a["w"], a["dw"], a["T"], a["E"], a["k"], 0.1,
                                        a["rule"], None) == EINVAL, bad


def test_more_tokens_than_indices_hold():
    L = k.lib()
    T = (1 << 30) + 1
    assert L.k3moe_swiglu_ckpt_bytes(T, 32) == -1
    assert L.k3moe_swiglu_forward(P, 32, P, 1 << 60, P, 32, P, 32, 0, T, 32, None) == EINVAL
    ws = L.k3moe_balance_workspace(32)
    assert L.k3moe_balance_forward(P, P, P, P, 0, 32, P, None, T, 32, 2, 0.1, 0, P, ws, None) == EINVAL
    assert L.k3moe_balance_backward(2 * P, 32, P, 0, 32, P, None, P, P, P, None, None, T, 32, 2, 0.1, 0, None) == EINVAL


def test_binding_refuses_other_tensors():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        k._dtype(x.half())
    with pytest.raises(TypeError):
        k._dtype(x, x.bfloat16())
    with pytest.raises(ValueError):
        k._ld(x.t(), 8, 4)
    with pytest.raises(ValueError):
        k._ld(x, 4, 7)
    with pytest.raises(ValueError):
        k._flat(x.t(), torch.float32, 8, 4)
    with pytest.raises(ValueError):
        k._flat(x, torch.int32, 4, 8)
    assert k._ld(x[:1, :3], 1, 3) == 8 and k._ld(x[:, :1], 4, 1) == 8


def test_operand_codes_of_the_wrong_size():
    """Codes given by the caller are the operand's bytes, all of them."""
    torch = pytest.importorskip("torch")
    ok = k.MxOperand(3, 33, codes=torch.empty(3, 32, dtype=torch.uint8))
    assert ok.atoms.numel() == k.lib().k3moe_mx_operand_atoms_bytes(3, 33)
    for bad in (torch.empty(3, 31, dtype=torch.uint8), torch.empty(3, 32, dtype=torch.int8),
                torch.empty(32, 3, dtype=torch.uint8).t(), torch.empty(0, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            k.MxOperand(3, 33, codes=bad)
