"""The operators together, as examples/train_moe.py runs them: a block's output and all
its gradients against the same steps in fp64, and the run as a captured graph."""
import os
import sys

import numpy as np
import pytest
import torch

import e4m3_reference as ref
import mx_reference as mx
from conftest import ROOT
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))
import train_moe  # noqa: E402


def _f64(t):
    return t.detach().double().cpu().numpy()


def _bf16(v):
    return torch.from_numpy(np.asarray(v, np.float64)).float().bfloat16().double().numpy()


def _q8(v):
    return ref.quantize(np.asarray(v, np.float32))[0]


def _near(got, want):
    """The same to 5e-3 of the norm.  Both sides round at the same places; what differs is
    values next to a rounding border: of bf16 results 2^-20 / 2^-8 or so take the other
    neighbour, 2^-8 away (6e-5 of a norm), of 8-bit ones as many and those whose input did,
    2^-4 away (3e-4), over six steps one after the other below 3e-3."""
    got, want = _f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape
    assert np.linalg.norm(got - want) <= 5e-3 * np.linalg.norm(want)


def _reference(b, x, delta, dout, dr):
    """Forward and backward of the block in fp64 with the same quantisation, on the
    router's choice as the block made it."""
    T, E, kk = b.T, b.E, b.top_k
    W = {n: np.stack([mx.values(*mx.quantize(_f64(w))) for w in p.W]) for n, p in
         (("gate", b.gate), ("up", b.up), ("down", b.down))}
    Wt = {n: np.stack([mx.values(*mx.quantize(_f64(w).T)) for w in p.W]) for n, p in
          (("gate", b.gate), ("up", b.up), ("down", b.down))}
    ids, w = b.ids.cpu().numpy(), _f64(b.w)
    off, order, pos = ref.plan(ids, E)
    tok = order // kk
    groups = [slice(off[e], off[e + 1]) for e in range(E)]

    def product(A, mats, rows):
        out = np.zeros((T * kk, mats.shape[1]))
        for e, s in enumerate(groups):
            out[s] = A[rows[s]] @ mats[e].T
        return out
    o, at = {}, np.arange(T * kk)
    r = _bf16(_f64(x) + _f64(delta))
    s = 1 / np.sqrt((r * r).mean(1, keepdims=True) + 1e-6)
    gain = _f64(b.gain)
    u, u8 = _bf16(r * s * gain), _q8(r * s * gain)
    g, v = _bf16(product(u8, W["gate"], tok)), _bf16(product(u8, W["up"], tok))
    h = _bf16(g / (1 + np.exp(-g)) * v)
    y = _bf16(product(_q8(h), W["down"], at))
    o["out"] = np.einsum("tkn,tk->tn", y[pos].reshape(T, kk, -1), w)
    # backward
    D = _f64(dout)
    dy = _bf16(w.reshape(-1)[order][:, None] * D[tok])
    dw = np.einsum("tkn,tn->tk", y[pos].reshape(T, kk, -1), D)
    dh = _bf16(product(_q8(dy), Wt["down"], at))
    gk, vk = _q8(g), _q8(v)
    sg = 1 / (1 + np.exp(-gk))
    dg, dv = _bf16(dh * vk * sg * (1 + gk * (1 - sg))), _bf16(dh * gk * sg)
    dslots = product(_q8(dg), Wt["gate"], at) + product(_q8(dv), Wt["up"], at)
    o["down"] = np.stack([dy[s].T @ h[s] for s in groups])
    o["gate"] = np.stack([dg[s].T @ u[tok[s]] for s in groups])
    o["up"] = np.stack([dv[s].T @ u[tok[s]] for s in groups])
    # router: softmax weights of the chosen, and the balance loss
    R = _f64(b.router)
    logits = u @ R.T
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    fr = E * np.bincount(ids.reshape(-1), minlength=E) / (kk * T)
    dl = 0.01 / T * p * (fr - (p @ fr)[:, None])
    inner = (w * dw).sum(1, keepdims=True)
    for j in range(kk):
        dl[np.arange(T), ids[:, j]] += w[:, j] * (dw[:, j] - inner[:, 0])
    o["router"] = dl.T @ u
    du = dl @ R + dslots[pos].reshape(T, kk, -1).sum(1)
    du = _bf16(du)
    xh, gg = r * s, du * gain
    o["gain"] = (du * xh).sum(0)
    o["dx"] = s * (gg - xh * (gg * xh).mean(1, keepdims=True)) + _f64(dr)
    return o


@pytest.mark.parametrize("T,d,f,E,kk", [(60, 256, 128, 6, 2), (1, 128, 128, 4, 4), (333, 384, 256, 5, 3), (700, 128, 256, 3, 1)])
def test_block_forward_and_gradients(T, d, f, E, kk):
    b = train_moe.MoeBlock(T, d, f, E, kk, seed=T)
    gen = torch.Generator(device="cuda").manual_seed(T)
    t = lambda s: (torch.randn(T, d, generator=gen, device="cuda") * s).bfloat16()  # noqa: E731
    b.gain.uniform_(0.5, 1.5, generator=gen)
    x, delta, dout, dr = t(1.0), t(0.5), t(0.1), t(0.1)
    b.quantize()
    b.forward(x, delta)
    b.backward(dout, dr)
    assert k.device_error() == 0
    want = _reference(b, x, delta, dout, dr)
    for got, name in ((b.out, "out"), (b.gate.dW, "gate"), (b.up.dW, "up"), (b.down.dW, "down"), (b.drouter, "router"),
                      (b.dgain, "gain"), (b.dx, "dx")):
        _near(got, want[name])


def test_block_as_a_graph():
    """Forward and backward captured once and replayed on new inputs and weights."""
    T, d, f, E, kk = 128, 256, 128, 8, 2
    b = train_moe.MoeBlock(T, d, f, E, kk, seed=3)
    eager = train_moe.MoeBlock(T, d, f, E, kk, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ins = [(torch.randn(T, d, generator=gen, device="cuda") * s).bfloat16() for s in (1.0, 0.5, 0.1, 0.1)]

    def run(b, x, delta, dout, dr):
        b.quantize()
        b.forward(x, delta)
        b.backward(dout, dr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(b, *ins)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, *ins)
    for i in range(3):
        for t in ins:
            t.copy_(torch.randn(T, d, generator=gen, device="cuda").bfloat16())
        for p, q in ((b.gate, eager.gate), (b.up, eager.up), (b.down, eager.down)):
            p.W.mul_(1.1 + i)
            q.W.copy_(p.W)
        graph.replay()
        run(eager, *ins)
        torch.cuda.synchronize()
        for name in ("out", "dx", "dgain", "dw", "r", "u", "ids"):
            assert torch.equal(getattr(b, name), getattr(eager, name)), name
        for p, q in ((b.gate, eager.gate), (b.up, eager.up), (b.down, eager.down)):
            assert torch.equal(p.dW, q.dW)
    assert k.device_error() == 0


def test_example_runs():
    losses, block = train_moe.train(steps=5)
    assert len(losses) == 5 and np.isfinite(losses).all()
    assert int(block.counts.sum()) == 512 * 4 and k.device_error() == 0
