"""SwiGLU and its gradients at gates far from zero, where sigma is below the
smallest normal fp32 number but the product is not, and over more chunks than the
grid takes in one step."""
import numpy as np
import pytest
import torch

import test_gpu_swiglu as base
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT, HALF = base.DT, base.HALF
# e^(-|g|/2) (2 ulp, 2^-22 each) twice, 1 / (1 + e^-|g|) (at most 7 steps of 2^-24), four products
REL = 24 * 2.0 ** -24


def _rows(dt):
    """Gates from -170 to 170, each with an `up` that makes g sigma(g) u a number of
    ordinary size where fp32 can hold one; the last rows mix such gates with small ones."""
    g = np.concatenate([np.linspace(-170, 170, 64 * 40), np.linspace(-100, -80, 64 * 8)]).reshape(-1, 64)
    mixed = np.random.default_rng(1).standard_normal((8, 64))
    mixed[:, ::9] = -95.0
    mixed[:, 40] = 88.5
    g = np.concatenate([g, mixed])
    u = np.exp(np.clip(-g, -5, 85)) * np.where(np.arange(64) % 2, -0.75, 1.25)
    return (torch.from_numpy(a.astype(np.float32)).to(DT[dt]).cuda() for a in (g, u))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gates_far_out(dt):
    g, u = _rows(dt)
    T, f = g.shape
    ck, h = k.SwigluCheckpoint(T, f), torch.empty_like(g)
    k.swiglu_forward(h, ck, g, u)
    G, U = base._f64(g), base._f64(u)
    want = G * base._sigma(G) * U
    tiny = 2.0 ** -126  # results below the smallest normal number have fewer digits
    assert (np.abs(base._f64(h) - want) <= np.abs(want) * (REL + HALF[dt]) + tiny).all()
    assert (np.abs(want[(G < -88) & (G > -150)]) > 1e-10).any()
    G, U = base._check_ckpt(ck, G, U)
    for scale in (1e-3, 1e3):
        dh = torch.full_like(g, scale)
        dg, du = torch.empty_like(g), torch.empty_like(g)
        k.swiglu_backward(dg, du, dh, ck)
        D, s = base._f64(dh), base._sigma(G)
        want_u = D * G * s
        assert (np.abs(base._f64(du) - want_u) <= np.abs(want_u) * (REL + HALF[dt]) + tiny).all()
        want_g = D * U * s * (1 + G * (1 - s))
        # 1 - sigma and the sum with 1 lose 2^-24 of their own size before they cancel
        slack = np.abs(D * U * s) * (1 + 2 * np.abs(G)) * REL
        assert (np.abs(base._f64(dg) - want_g) <= slack + np.abs(want_g) * HALF[dt] + tiny).all()


# 152 SMs x 48 runs x 256 threads take 1.87 million chunks of eight values a step
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,f", [(4001, 4096), (12001, 4096), (4001, 4001), (9001, 4001), (70001, 250)])
def test_many_chunks_a_thread(T, f, dt):
    """Against the same rows in small calls, bit for bit, for whole aligned chunks
    and for rows that are not made of them."""
    gen = torch.Generator(device="cuda").manual_seed(T + f)
    g, u, dh = (torch.randn(T, f, generator=gen, device="cuda").to(DT[dt]) for _ in range(3))
    ck, h, dg, du = k.SwigluCheckpoint(T, f), torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    k.swiglu_forward(h, ck, g, u)
    k.swiglu_backward(dg, du, dh, ck)
    pad = -(-f // 32) * 32
    codes = ck.data[:2 * T * pad].view(2, T, pad)
    scales = ck.data[2 * T * pad:].view(2, T, pad // 32)
    step = 997
    for a in range(0, T, step):
        b = min(T, a + step)
        n = b - a
        c, hh, dgg, duu = k.SwigluCheckpoint(n, f), torch.empty_like(g[a:b]), torch.empty_like(g[a:b]), torch.empty_like(g[a:b])
        k.swiglu_forward(hh, c, g[a:b], u[a:b])
        k.swiglu_backward(dgg, duu, dh[a:b], c)
        assert torch.equal(h[a:b], hh) and torch.equal(dg[a:b], dgg) and torch.equal(du[a:b], duu), a
        assert torch.equal(codes[:, a:b], c.data[:2 * n * pad].view(2, n, pad))
        assert torch.equal(scales[:, a:b], c.data[2 * n * pad:].view(2, n, pad // 32))
