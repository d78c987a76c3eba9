"""A whole mixture-of-experts block, trained with the library's operators.

r = x + delta; u = norm(r); the router's choice of u; every expert's SwiGLU over its
tokens with MXFP4 matrices and 8-bit rows; the weighted sum of each token's experts.
Backward: the same matrices transposed for the input gradients (8-bit rows again),
bf16 rows for the weight gradients, the balance loss and the combine weights for the
router, the norm for the stream.  The products, weight gradients and combines are one
call each for all experts; the weights' operands are made anew in every step, a call for
each expert's matrix.

    python examples/train_moe.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mxfp4_routed_expert_select_gb300 import k3moe as k  # noqa: E402


class MoeLinear:
    """The matrices [E][n][m] of one projection: fp32 masters, MXFP4 operands for the
    output and (transposed) for the input gradient."""

    def __init__(self, E, n, m, gen):
        self.W = torch.randn(E, n, m, generator=gen, device="cuda") * m ** -0.5
        self.dW = torch.empty_like(self.W)
        self.fwd, self.bwd = k.MxExperts(E, n, m), k.MxExperts(E, m, n)

    def quantize(self):
        for e in range(self.W.shape[0]):
            k.mx_quantize_operand(self.W[e], self.fwd.operand(e), self.bwd.operand(e))


class MoeBlock:
    """T tokens of width d, E experts of size f, top_k of them for a token.  d and f are
    multiples of 128."""

    def __init__(self, T, d, f, E, top_k, seed=0, alpha=0.01):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.E, self.top_k = T, E, top_k
        self.gate, self.up, self.down = MoeLinear(E, f, d, gen), MoeLinear(E, f, d, gen), MoeLinear(E, d, f, gen)
        self.gain = torch.ones(d, device="cuda")
        self.router = (torch.randn(E, d, generator=gen, device="cuda") * d ** -0.5).bfloat16()
        self.layer = k.Layer(E, top_k, d, f, self.router.view(torch.int16), None, max_tokens=T)
        self.norm, self.groups = k.RmsNorm(d, 1e-6), k.ExpertGroups(E, top_k, T)
        self.balance = k.BalanceLoss(E, top_k, alpha)
        S = T * top_k
        new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        f32, i32 = torch.float32, torch.int32
        self.r, self.u, self.u8, self.rstd = new(T, d), new(T, d), k.Mx8Rows(T, d), new(T, dtype=f32)
        self.ids, self.w = new(T, top_k, dtype=i32), new(T, top_k, dtype=f32)
        self.g, self.v, self.h, self.h8 = new(S, f), new(S, f), new(S, f), k.Mx8Rows(S, f)
        self.y, self.out, self.ckpt = new(S, d), new(T, d), k.SwigluCheckpoint(S, f)
        self.loss, self.counts, self.valid = new(1, dtype=f32), new(E, dtype=i32), new(1, dtype=i32)
        # backward
        self.dy, self.dw, self.dy8 = new(S, d), new(T, top_k, dtype=f32), k.Mx8Rows(S, d)
        self.dh, self.dg, self.dv, self.dg8, self.dv8 = new(S, f), new(S, f), new(S, f), k.Mx8Rows(S, f), k.Mx8Rows(S, f)
        self.dslots, self.du, self.dlogits = new(S, d, dtype=f32), new(T, d, dtype=f32), new(T, E, dtype=f32)
        self.dx, self.dgain, self.drouter = new(T, d), new(d, dtype=f32), new(E, d, dtype=f32)
        self.one = torch.ones(1, device="cuda")

    def quantize(self):
        """The operands of the weights as they are now."""
        for p in (self.gate, self.up, self.down):
            p.quantize()

    def forward(self, x, delta):
        """x, delta bf16 [T][d] -> what the block adds to the stream self.r = x + delta."""
        self.norm.forward(self.u, x, delta, self.r, self.rstd, self.gain, self.u8)
        self.layer.route(self.u, self.T, self.ids, self.w)
        self.logits = self.u.float() @ self.router.float().t()
        self.balance.forward(self.loss, self.counts, self.valid, self.logits, self.ids)
        self.groups.plan(self.ids)
        k.grouped_matmul(self.g, self.u8, self.gate.fwd, self.groups, gather=True)
        k.grouped_matmul(self.v, self.u8, self.up.fwd, self.groups, gather=True)
        k.swiglu_forward(self.h, self.ckpt, self.g, self.v)
        k.mx8_quantize(self.h8, self.h)
        k.grouped_matmul(self.y, self.h8, self.down.fwd, self.groups)
        k.combine(self.out, self.y, self.groups, self.w)
        return self.out

    def backward(self, dout, dr=None):
        """dout of the block's output, dr of the stream -> dx (of x and of delta)."""
        k.combine_backward(self.dy, self.dw, dout, self.y, self.groups, self.w)
        k.mx8_quantize(self.dy8, self.dy)
        k.grouped_matmul(self.dh, self.dy8, self.down.bwd, self.groups)
        k.grouped_wgrad(self.down.dW, self.dy, self.h, self.groups)
        k.swiglu_backward(self.dg, self.dv, self.dh, self.ckpt)
        k.mx8_quantize(self.dg8, self.dg)
        k.mx8_quantize(self.dv8, self.dv)
        k.grouped_matmul(self.dslots, self.dg8, self.gate.bwd, self.groups)
        k.grouped_matmul(self.dslots, self.dv8, self.up.bwd, self.groups, accumulate=True)
        k.grouped_wgrad(self.gate.dW, self.dg, self.u, self.groups, gather=True)
        k.grouped_wgrad(self.up.dW, self.dv, self.u, self.groups, gather=True)
        # the router: its balance loss and the gradient of the combine weights
        self.balance.backward(self.dlogits, self.logits, self.ids, self.counts, self.valid, self.one, None, self.w, self.dw)
        torch.matmul(self.dlogits.t(), self.u.float(), out=self.drouter)
        torch.matmul(self.dlogits, self.router.float(), out=self.du)
        k.combine(self.du, self.dslots, self.groups, accumulate=True)
        self.norm.backward(self.dx, self.dgain, self.du.bfloat16(), self.r, self.rstd, self.gain, dr)
        return self.dx

    def step(self, lr):
        for p in (self.gate, self.up, self.down):
            p.W.sub_(p.dW, alpha=lr)
        self.gain.sub_(self.dgain, alpha=lr)
        self.router.sub_((self.drouter * lr).bfloat16())


def train(steps=50, T=512, d=256, f=128, E=16, top_k=4, seed=0, lr=0.5):
    """Fits the block to a fixed map of its input; returns the losses and the block."""
    block = MoeBlock(T, d, f, E, top_k, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    A = randn(d, d) * d ** -0.5
    losses = []
    for _ in range(steps):
        x, delta = randn(T, d).bfloat16(), (randn(T, d) * 0.5).bfloat16()
        block.quantize()
        out = block.forward(x, delta).float()
        diff = out - torch.tanh((x + delta).float() @ A)
        losses.append(float(diff.square().mean()))
        block.backward((diff / T).bfloat16())
        block.step(lr)
    return losses, block


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=50)
    losses, block = train(ap.parse_args().steps)
    print("loss first %.4f  last %.4f" % (losses[0], losses[-1]))
    print("tokens an expert min %d  max %d" % (int(block.counts.min()), int(block.counts.max())))
