"""One MXFP4 expert and a router, trained with the library's operators.

The expert y = W_down (silu(W_gate x) * (W_up x)) learns a teacher's outputs with
every product in MXFP4 (forward, input gradients, weight gradients) and its SwiGLU
kept in 8 bits; the router's weights follow the balance loss until its experts are
chosen evenly.  At the end the trained expert is packed as the layer stores it and
run by the batch-1 call.

    python examples/train_expert.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mxfp4_routed_expert_select_gb300 import k3moe as k  # noqa: E402


class MxLinear:
    """y = x W^T in MXFP4 with an fp32 master weight W [n][m]."""

    def __init__(self, n, m, T, scale, gen):
        self.W = torch.randn(n, m, generator=gen, device="cuda") * scale
        self.dW = torch.empty_like(self.W)
        self.wr, self.wc = k.MxOperand(n, m), k.MxOperand(m, n)
        self.xr, self.xc = k.MxOperand(T, m), k.MxOperand(m, T)
        self.gr, self.gc = k.MxOperand(T, n), k.MxOperand(n, T)

    def forward(self, y, x):
        k.mx_quantize_operand(self.W, self.wr, self.wc)
        k.mx_quantize_operand(x, self.xr, self.xc)
        k.mx_matmul(y, self.xr, self.wr)

    def backward(self, dx, dy, accumulate=False):
        k.mx_quantize_operand(dy, self.gr, self.gc)
        k.mx_matmul(dx, self.gr, self.wc, accumulate)
        k.mx_matmul(self.dW, self.gc, self.xc)

    def step(self, lr):
        self.W.sub_(self.dW, alpha=lr)


class Expert:
    """A SwiGLU expert of T tokens a step."""

    def __init__(self, d, f, T, gen):
        self.gate, self.up = MxLinear(f, d, T, d ** -0.5, gen), MxLinear(f, d, T, d ** -0.5, gen)
        self.down = MxLinear(d, f, T, f ** -0.5, gen)
        new = lambda n: torch.empty(T, n, device="cuda")  # noqa: E731
        self.g, self.u, self.h, self.y, self.dx = new(f), new(f), new(f), new(d), new(d)
        self.ckpt = k.SwigluCheckpoint(T, f)

    def forward(self, x):
        self.gate.forward(self.g, x)
        self.up.forward(self.u, x)
        k.swiglu_forward(self.h, self.ckpt, self.g, self.u)
        self.down.forward(self.y, self.h)
        return self.y

    def backward(self, dy):
        dh = self.h  # the forward value is not needed any more
        self.down.backward(dh, dy)
        k.swiglu_backward(self.g, self.u, dh, self.ckpt)
        self.gate.backward(self.dx, self.g)
        self.up.backward(self.dx, self.u, accumulate=True)
        return self.dx

    def step(self, lr):
        for p in (self.gate, self.up, self.down):
            p.step(lr)

    def packed(self, d, f):
        """The weights as the layer stores them (six MXFP4 planes in one blob)."""
        planes = {}
        for name, p in (("gate", self.gate), ("up", self.up), ("down", self.down)):
            n, m = p.W.shape
            codes = torch.empty(n, m // 2, dtype=torch.uint8, device="cuda")
            scales = torch.empty(n, m // 32, dtype=torch.uint8, device="cuda")
            k.mx_quantize(codes, scales, p.W, n, m)
            planes[name + "_packed"], planes[name + "_scales"] = codes, scales
        blob = torch.empty(k.expert_bytes(d, f), dtype=torch.uint8, device="cuda")
        k.pack_expert(blob, planes, d, f)
        return blob


def train(steps=200, d=512, f=256, T=512, E=32, top_k=4, seed=0, lr=0.05):
    """Returns the expert's losses, the balance losses, the last counts, and the
    batch-1 call's output of the trained expert beside the training forward's."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    student = Expert(d, f, T, gen)
    tg, tu, td = randn(f, d) * d ** -0.5, randn(f, d) * d ** -0.5, randn(d, f) * f ** -0.5

    # a router that starts out favouring some experts: a direction all tokens share
    common = randn(d)
    Wr = randn(E, d) * 0.05 + randn(E, 1) * common * 0.002
    ids, w = torch.empty(T, top_k, dtype=torch.int32, device="cuda"), torch.empty(T, top_k, device="cuda")
    loss, dloss = torch.empty(1, device="cuda"), torch.ones(1, device="cuda")
    counts, valid = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    dlogits, dWr = torch.empty(T, E, device="cuda"), torch.empty(E, d, device="cuda")
    balance = k.BalanceLoss(E, top_k, alpha=1.0)
    gl, xl = k.MxOperand(E, T), k.MxOperand(d, T)

    losses, balances = [], []
    for _ in range(steps):
        x = randn(T, d) + common * 0.5
        # the expert
        want = (torch.nn.functional.silu(x @ tg.t()) * (x @ tu.t())) @ td.t()
        diff = student.forward(x) - want
        losses.append(float(diff.square().mean()))
        student.backward(diff / T)
        student.step(lr)
        # the router: the layer's own selection, the balance loss of its choice
        bits = Wr.bfloat16()
        router = k.Layer(E, top_k, d, f, bits.view(torch.int16), None, max_tokens=T)
        router.route(x, T, ids, w)
        logits = x @ bits.float().t()
        balance.forward(loss, counts, valid, logits, ids)
        balance.backward(dlogits, logits, ids, counts, valid, dloss)
        k.mx_quantize_operand(dlogits, None, gl)
        k.mx_quantize_operand(x, None, xl)
        k.mx_matmul(dWr, gl, xl)
        Wr.sub_(dWr, alpha=0.05)
        balances.append(float(loss))
        router.close()

    blob = student.packed(d, f)
    expert = k.expert_view(blob.data_ptr(), d, f)
    y = torch.empty(d, device="cuda")
    ws = torch.empty(k.expert_gemv_workspace(d, f), dtype=torch.uint8, device="cuda")
    k.expert_gemv(y, x[0].contiguous(), expert, d, f, ws)
    return losses, balances, counts.cpu(), (y, student.forward(x)[0])


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    losses, balances, counts, (y, z) = train(ap.parse_args().steps)
    print("expert loss      first %.4f  last %.4f" % (losses[0], losses[-1]))
    print("balance loss     first %.4f  last %.4f (1 is even)" % (balances[0], balances[-1]))
    print("tokens an expert min %d  max %d" % (counts.min(), counts.max()))
    print("batch-1 call against the training forward (its activations in MXFP4): relative %.3f"
          % float((y - z).norm() / y.norm()))
