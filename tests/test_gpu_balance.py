"""The router's balance loss: counts, loss and the gradient of the logits against
fp64 formulas and against differences, over the three rules, masks, dropped
slots, experts masked to -inf, sizes and types."""
import numpy as np
import pytest
import torch

from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
RULES = ["softmax", "sigmoid", "sigmoid_norm"]
ALPHA = 0.02


def _probs(l, rule):
    """(p, 1 - sigma) of fp64 logits, rows of -inf entries included."""
    if rule == "softmax":
        x = np.exp(l - l.max(1, keepdims=True))
        return x / x.sum(1, keepdims=True), None
    m = np.minimum(l.max(1, keepdims=True), 0)
    with np.errstate(over="ignore"):
        x = np.where(l > 0, 1 / (1 + np.exp(-l)), np.exp(l - m) / (1 + np.exp(np.minimum(l, 0))))
        r = 1 / (1 + np.exp(l))
    return x / x.sum(1, keepdims=True), r


def formula(l, ids, mask, rule, dloss, w, dw):
    T, E = l.shape
    K = ids.shape[1]
    on = (l > -np.inf).any(1)
    if mask is not None:
        on &= mask != 0
    n = int(on.sum())
    slot = (ids >= 0) & (ids < E) & on[:, None]
    counts = np.bincount(ids[slot], minlength=E)
    grad = np.zeros_like(l)
    if n == 0:
        return 0.0, counts, n, grad, np.zeros_like(l)
    p, r = _probs(l[on], rule)
    f = counts * E / (K * n)
    loss = ALPHA * (f * p.mean(0)).sum()
    f1 = (counts * E - K * n) / (K * n)  # f - 1: the same differences, exactly 0 for an even choice
    g = ALPHA * dloss / n * p * (f1 - (p @ f1)[:, None])
    size = ALPHA * abs(dloss) / n * p * (np.abs(f - 1) + (p @ np.abs(f - 1))[:, None])
    if rule != "softmax":
        g, size = g * r, size * r
    grad[on] = g
    mag = np.zeros_like(l)
    mag[on] = size
    if w is not None:
        inner = (w * dw * slot).sum(1, keepdims=True)
        inner_abs = (w * np.abs(dw) * slot).sum(1, keepdims=True)
        for t, j in zip(*np.nonzero(slot)):
            x = l[t, ids[t, j]]
            s, rr = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
            if rule == "softmax":
                c, a = w[t, j] * (dw[t, j] - inner[t, 0]), w[t, j] * (abs(dw[t, j]) + inner_abs[t, 0])
            elif rule == "sigmoid":
                c = s * rr * dw[t, j]
                a = abs(c)
            else:
                c, a = w[t, j] * rr * (dw[t, j] - inner[t, 0]), w[t, j] * rr * (abs(dw[t, j]) + inner_abs[t, 0])
            grad[t, ids[t, j]] += c
            mag[t, ids[t, j]] += a
    return loss, counts, n, grad, mag


def make(T, E, K, rule, dt, seed, masked=0.0, dropped=0.0, weights=True, ninf=0.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E + pad, generator=g) * 2 + torch.randn(E + pad, generator=g)
    if ninf:
        l[torch.rand(T, E + pad, generator=g) < ninf] = float("-inf")
        l[0] = float("-inf")
    l = l.to(DT[dt])
    ids = torch.topk(l[:, :E].float(), K, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, K, generator=g) < dropped] = -1
    mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
    w = torch.rand(T, K, generator=g) if weights else None
    dw = torch.randn(T, K, generator=g) * 0.1 if weights else None
    return l.cuda()[:, :E], ids.cuda(), None if mask is None else mask.cuda(), \
        None if w is None else w.cuda(), None if dw is None else dw.cuda()


def call(l, ids, mask, rule, dloss, w, dw, bal=None, alpha=ALPHA):
    T, E = l.shape
    bal = bal or k.BalanceLoss(E, ids.shape[1], alpha, rule)
    loss, counts = torch.full((1,), 7.0, device="cuda"), torch.full((E,), -5, dtype=torch.int32, device="cuda")
    n = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    dl = torch.full((T, E), 3.0, dtype=l.dtype, device="cuda")
    d = torch.full((1,), dloss, device="cuda")
    bal.forward(loss, counts, n, l, ids, mask)
    bal.backward(dl, l, ids, counts, n, d, mask, w, dw)
    torch.cuda.synchronize()
    assert not bool(bal.workspace.any()), "the workspace is left zero"
    return loss, counts, n, dl


def compare(l, ids, mask, rule, dloss, w, dw, got):
    c = lambda t: None if t is None else t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    idn = ids.cpu().numpy().astype(np.int64)
    loss, counts, n, grad, mag = formula(c(l), idn, None if mask is None else mask.cpu().numpy(), rule, dloss, c(w), c(dw))
    g_loss, g_counts, g_n, g_dl = got
    T, E = l.shape
    assert int(g_n) == n
    assert np.array_equal(g_counts.cpu().numpy(), counts)
    # p: exp and division within 4 ulp, a row's sum within log2(E) + 32 steps;
    # a warp adds at most T / 8 rows' p in fp32
    rel = (48 + T / 8) * 2.0 ** -24
    assert abs(float(g_loss) - loss) <= rel * abs(loss) + 1e-12
    # the gradient: p as above, <f - 1, p> in fp32 over E terms, a few products;
    # one rounding to the output type
    half = 2.0 ** -8 if l.dtype == torch.bfloat16 else 2.0 ** -24
    tol = mag * 96 * 2.0 ** -24 + np.abs(grad) * half + 1e-38
    err = np.abs(c(g_dl) - grad)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("T,E,K,masked,dropped,weights,ninf,pad",
                         [(1, 1, 1, 0, 0, True, 0, 0), (1, 896, 16, 0, 0, True, 0, 0), (7, 8, 8, 0, 0, False, 0, 1),
                          (64, 896, 16, 0.3, 0.1, True, 0, 0), (100, 33, 4, 0, 0.5, True, 0.3, 2),
                          (333, 130, 32, 0.5, 0, False, 0, 0), (500, 257, 6, 0, 0.2, True, 0.5, 0),
                          (2500, 600, 10, 0.1, 0.1, True, 0, 4), (31, 1024, 16, 0, 0, True, 0.9, 0)])
def test_loss_counts_gradient(T, E, K, masked, dropped, weights, ninf, pad, rule, dt):
    l, ids, mask, w, dw = make(T, E, K, rule, dt, T + E, masked, dropped, weights, ninf, pad)
    compare(l, ids, mask, rule, 1.5, w, dw, call(l, ids, mask, rule, 1.5, w, dw))


@pytest.mark.parametrize("rule", RULES)
def test_no_valid_token(rule):
    l, ids, _, w, dw = make(20, 40, 4, rule, "f32", 3)
    mask = torch.zeros(20, dtype=torch.uint8, device="cuda")
    for ll, m in ((l, mask), (torch.full_like(l, float("-inf")), None)):
        loss, counts, n, dl = call(ll, ids, m, rule, 1.0, w, dw)
        assert float(loss) == 0 and int(n) == 0 and not bool(counts.any()) and not bool(dl.any())


def test_masked_tokens_may_hold_anything():
    l, ids, _, w, dw = make(30, 50, 4, "softmax", "f32", 4)
    mask = torch.ones(30, dtype=torch.uint8, device="cuda")
    mask[::3] = 0
    want = call(l, ids, mask, "softmax", 1.0, w, dw)
    l2, w2, dw2, ids2 = l.clone(), w.clone(), dw.clone(), ids.clone()
    l2[::3] = float("nan")
    l2[0] = float("inf")
    w2[::3] = dw2[::3] = float("nan")
    ids2[::3] = 2 ** 30
    got = call(l2, ids2, mask, "softmax", 1.0, w2, dw2)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_logit_of_a_valid_token_shows(bad):
    l, ids, _, w, dw = make(30, 50, 4, "softmax", "f32", 4)
    l[11, 7] = bad
    loss, counts, n, dl = call(l, ids, None, "softmax", 1.0, w, dw)
    assert bool(torch.isnan(loss)) and int(n) == 30 and int(counts.sum()) == 120
    assert bool(torch.isnan(dl[11]).all()) and bool(torch.isfinite(dl[:11]).all())


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("level", [-300.0, -90.0, 90.0, 300.0])
def test_extreme_logits(rule, level):
    l, ids, _, w, dw = make(16, 70, 5, rule, "f32", 9)
    l = l + level
    compare(l, ids, None, rule, 1.0, w, dw, call(l, ids, None, rule, 1.0, w, dw))


@pytest.mark.parametrize("rule", RULES)
def test_gradient_against_differences(rule):
    """Central differences of loss + <dw, w(l)> in fp64, counts held."""
    T, E, K = 6, 24, 4
    l, ids, _, _, dw = make(T, E, K, rule, "f32", 12)
    L, idn, D = l.cpu().numpy().astype(np.float64), ids.cpu().numpy().astype(np.int64), dw.cpu().numpy().astype(np.float64)

    def weights(L):
        c = np.take_along_axis(L, idn, 1)
        if rule == "softmax":
            x = np.exp(c - c.max(1, keepdims=True))
            return x / x.sum(1, keepdims=True)
        s = 1 / (1 + np.exp(-c))
        return s if rule == "sigmoid" else s / s.sum(1, keepdims=True)

    f = np.bincount(idn.ravel(), minlength=E) * E / (K * T)

    def total(L):
        return ALPHA * (f * _probs(L, rule)[0].mean(0)).sum() + (D * weights(L)).sum()
    w = torch.from_numpy(weights(L).astype(np.float32)).cuda()
    dl = call(l, ids, None, rule, 1.0, w, dw)[3].cpu().numpy()
    h = 1e-4
    for t in range(T):
        for e in range(0, E, 5):
            up, dn = L.copy(), L.copy()
            up[t, e] += h
            dn[t, e] -= h
            num = (total(up) - total(dn)) / (2 * h)
            assert abs(dl[t, e] - num) <= 1e-8 + 2e-6 * np.abs(D).max()


def test_repeated_ids_and_in_place():
    """Slots that name one expert more than once add up; dlogits may be logits."""
    l, ids, _, w, dw = make(40, 30, 6, "softmax", "f32", 15)
    ids[:, 3] = ids[:, 1]
    ids[:, 5] = ids[:, 1]
    got = call(l, ids, None, "softmax", 1.0, w, dw)
    compare(l, ids, None, "softmax", 1.0, w, dw, got)
    bal, d = k.BalanceLoss(30, 6, ALPHA), torch.ones(1, device="cuda")
    for rule in RULES:
        bal = k.BalanceLoss(30, 6, ALPHA, rule)
        want = call(l, ids, None, rule, 1.0, w, dw)
        x = l.clone()
        bal.backward(x, x, ids, want[1], want[2], d, None, w, dw)
        assert torch.equal(x, want[3])


def test_repeats_bit_for_bit_and_from_a_graph():
    l, ids, mask, w, dw = make(3000, 200, 8, "softmax", "f32", 16, masked=0.2)
    bal = k.BalanceLoss(200, 8, ALPHA)
    first = call(l, ids, mask, "softmax", 1.0, w, dw, bal)
    for _ in range(4):
        for a, b in zip(first, call(l, ids, mask, "softmax", 1.0, w, dw, bal)):
            assert torch.equal(a, b)
    loss, counts, n, dl = (torch.zeros_like(t) for t in first)
    d = torch.ones(1, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bal.forward(loss, counts, n, l, ids, mask)
        bal.backward(dl, l, ids, counts, n, d, mask, w, dw)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (loss, counts, n, dl)):
        assert torch.equal(a, b)
