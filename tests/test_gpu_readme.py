"""The README's sequence for every expert's matrices, run as it stands there: its
outputs and its weight gradients against the fp64 definitions of what it says."""
import os
import re

import numpy as np
import pytest
import torch

import e4m3_reference as ref
import mx_reference as mx
from conftest import ROOT
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu


def _block(of):
    with open(os.path.join(ROOT, "README.md")) as fh:
        for code in re.findall(r"```python\n(.*?)```", fh.read(), re.S):
            if of in code:
                return code
    raise AssertionError("the README has no sequence with " + of)


def test_every_experts_matrices():
    T, K, N, E, top_k = 48, 256, 136, 6, 2
    gen = torch.Generator().manual_seed(3)
    rng = np.random.default_rng(3)
    t = lambda *s, scale=1.0: (torch.randn(*s, generator=gen) * scale).bfloat16().cuda()  # noqa: E731
    new = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ids = rng.integers(0, E, (T, top_k)).astype(np.int32)
    packed = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    scales = rng.integers(120, 128, (E, N, K // 32), dtype=np.uint8)
    names = dict(k=k, T=T, K=K, N=N, E=E, top_k=top_k, x=t(T, K, scale=2.0), delta=t(T, K), r=new(T, K), u=new(T, K),
                 gain=(1 + torch.randn(K, generator=gen) * 0.3).cuda(), ids=torch.from_numpy(ids).cuda(),
                 packed=torch.from_numpy(packed).cuda(), scales=torch.from_numpy(scales).cuda(), C=new(T * top_k, N),
                 out=new(T, N), w=torch.rand(T, top_k, generator=gen).cuda(), dC=new(T * top_k, N),
                 dw=torch.zeros(T, top_k, device="cuda"), dout=t(T, N), dW=torch.zeros(E, N, K, device="cuda"))
    x, delta = names["x"].clone(), names["delta"].clone()
    exec(_block("k.grouped_wgrad("), names)
    torch.cuda.synchronize()
    assert k.device_error() == 0
    f64 = lambda n: names[n].double().cpu().numpy()  # noqa: E731
    r = (x.float() + delta.float()).bfloat16().double().cpu().numpy()
    assert np.array_equal(f64("r"), r)
    u = r / np.sqrt((r * r).mean(1, keepdims=True) + 1e-6) * f64("gain")
    off, order, pos = ref.plan(ids, E)
    src = order // top_k  # every slot is kept
    V = np.stack([mx.values(mx.unpack(p), s) for p, s in zip(packed, scales)])
    A = ref.read_rows(names["x8"])[0]
    # 8-bit rows: a value to the nearest of the e4m3 codes at its block's scale, half a step
    # of 2^-3 or of the smallest code (2^-9) where the scale is at most max / 224
    top = np.abs(u).reshape(T, -1, 32).max(2).repeat(32, 1)
    assert (np.abs(A - u) <= np.abs(u) * 2.0 ** -4 * 1.001 + top / 224 * 2.0 ** -10 * 1.001).all()
    dC, dout, W = f64("dC"), f64("dout"), f64("w")
    for e in range(E):
        s = slice(off[e], off[e + 1])
        want, mag = A[src[s]] @ V[e].T, np.abs(A[src[s]]) @ np.abs(V[e]).T
        assert (np.abs(f64("C")[s] - want) <= mag * (K / 32 + 10) * 2.0 ** -22 + np.abs(want) * 2.0 ** -8).all()
        # the rows that made C, in bf16 (2^-8 of each); fp32 sums of 16 rows a step
        want, mag = dC[s].T @ u[src[s]], np.abs(dC[s]).T @ np.abs(u[src[s]])
        assert (np.abs(f64("dW")[e] - want) <= mag * (2.0 ** -8 + 2.0 ** -18) + 1e-30).all(), "gradient of expert %d" % e
    C = f64("C")[pos].reshape(T, top_k, N)
    want, mag = np.einsum("tkn,tk->tn", C, W), np.einsum("tkn,tk->tn", np.abs(C), W)
    assert (np.abs(f64("out") - want) <= np.abs(want) * 2.0 ** -8 + mag * 4 * 2.0 ** -24).all()
    want = np.zeros_like(dC)
    want[pos] = (W[..., None] * dout[:, None]).reshape(T * top_k, N)
    assert (np.abs(dC - want) <= np.abs(want) * 2.0 ** -8).all()
    want, mag = np.einsum("tkn,tn->tk", C, dout), np.einsum("tkn,tn->tk", np.abs(C), np.abs(dout))
    assert (np.abs(f64("dw") - want) <= mag * 32 * 2.0 ** -24).all()
