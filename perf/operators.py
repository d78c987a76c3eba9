"""The training and quantisation operators as measured cases.

Four operators around the MXFP4 routed-expert layer:

  quantise   an activation or weight matrix to MXFP4 along its rows, its
             columns, or both from one read
  product    C = A B^T of two MXFP4 matrices: the projection of a few tokens,
             of a batch, and one training step of an MXFP4 linear layer
             (output, input gradient, weight gradient)
  swiglu     h = silu(g) u with g and u kept for the backward pass as 8-bit
             block-scaled floats, and the gradients from those
  balance    the router's balance loss, the per-expert counts, and the
             gradient of the logits

`own` chooses between the plain forms (elementary torch operations in 32 bits)
and the library's calls.  A 4-bit operand is returned as the values it stands
for; an 8-bit checkpoint shows in the gradients computed from it.
"""
import torch

own = False

D, F, E, TOPK = 7168, 1536, 896, 16  # the layer's hidden and expert sizes, experts and experts per token


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one decode token on its way into an MXFP4 projection: launch latency
        dict(name="quantise_token", op="quantise", rows=1, cols=D, dtype="f32", along="rows"),
        # an expert's down weight turned to MXFP4 in both orientations for a training step
        dict(name="quantise_weight", op="quantise", rows=D, cols=F, dtype="bf16", along="both"),
        # a batch's activations, both orientations (forward product and weight gradient)
        dict(name="quantise_batch", op="quantise", rows=4096, cols=D, dtype="bf16", along="both"),
        # ragged gradient rows, fp32, columns only
        dict(name="quantise_ragged", op="quantise", rows=1003, cols=1537, dtype="f32", along="cols"),
        # serving: one token through one projection held in MXFP4 (weights streamed once)
        dict(name="product_token", op="product", M=1, N=D, K=F, dtype="f32"),
        # a decode batch through the gate-sized projection
        dict(name="product_tokens64", op="product", M=64, N=F, K=D, dtype="bf16"),
        # odd sizes in every direction
        dict(name="product_odd", op="product", M=333, N=1000, K=1112, dtype="f32"),
        # a training step of the gate projection at the prefill batch
        dict(name="linear_step", op="linear", T=4096, N=F, K=D, dtype="bf16"),
        # an expert's share of a decode batch, gate and up in one [T][2 f] tensor
        dict(name="swiglu_small", op="swiglu", T=64, f=F, dtype="bf16", fused=True),
        # every (token, expert) pair of a prefill batch
        dict(name="swiglu_pairs", op="swiglu", T=4096 * TOPK, f=F, dtype="bf16", fused=False),
        # the router of a decode batch
        dict(name="balance_small", op="balance", T=64, E=E, k=TOPK, dtype="f32", rule="softmax", masked=0.0,
             dropped=0.0, weights=True),
        # the router of a large training batch with padding tokens and dropped slots
        dict(name="balance_batch", op="balance", T=16384, E=E, k=TOPK, dtype="f32", rule="softmax", masked=0.1,
             dropped=0.02, weights=True),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantise", "product", "linear", "swiglu", "balance"])
    dt = rng.choice(["f32", "bf16"])
    if op == "quantise":
        rows, cols = _log_int(rng, 1, 4096), _log_int(rng, 17, D)
        return dict(op=op, rows=rows, cols=cols, dtype=dt, along=rng.choice(["rows", "cols", "both"]))
    if op == "product":
        return dict(op=op, M=_log_int(rng, 1, 4096), N=_log_int(rng, 24, D), K=_log_int(rng, 32, D), dtype=dt)
    if op == "linear":
        return dict(op=op, T=_log_int(rng, 16, 4096), N=_log_int(rng, 96, F), K=_log_int(rng, 96, D), dtype=dt)
    if op == "swiglu":
        return dict(op=op, T=_log_int(rng, 1, 32768), f=_log_int(rng, 40, F), dtype=dt, fused=rng.random() < 0.5)
    ne = _log_int(rng, 8, 1024)
    return dict(op=op, T=_log_int(rng, 1, 16384), E=ne, k=rng.randint(1, min(16, ne)), dtype=dt,
                rule=rng.choice(["softmax", "sigmoid", "sigmoid_norm"]), masked=rng.choice([0.0, 0.3]),
                dropped=rng.choice([0.0, 0.05]), weights=rng.random() < 0.7)


# -------------------------------------------------------------------- inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(case, seed):
    """The tensors a user's program has before the call, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    op = case["op"]
    if op == "quantise":
        # activations: normal values, a few channels an order of magnitude larger
        x = normal(case["rows"], case["cols"])
        x *= 1 + 15 * (torch.rand(case["cols"], generator=gen, device="cuda") < 0.01)
        return dict(x=x.to(dt))
    if op == "product":
        # weights as stored: random codes, scale exponents as in the layer's experts
        kp = -(-case["K"] // 32) * 32
        packed = torch.randint(0, 256, (case["N"], kp // 2), generator=gen, device="cuda", dtype=torch.uint8)
        if kp != case["K"]:  # codes past K are zero in a stored matrix
            tail = torch.arange(kp, device="cuda") < case["K"]
            packed &= (tail[0::2] * 15 + tail[1::2] * 240).to(torch.uint8)
        scales = torch.randint(120, 131, (case["N"], kp // 32), generator=gen, device="cuda", dtype=torch.uint8)
        return dict(x=normal(case["M"], case["K"]).to(dt), packed=packed, scales=scales)
    if op == "linear":
        return dict(x=normal(case["T"], case["K"]).to(dt), w=normal(case["N"], case["K"], scale=0.02).to(dt),
                    dy=normal(case["T"], case["N"], scale=1e-3).to(dt))
    if op == "swiglu":
        T, f = case["T"], case["f"]
        if case["fused"]:  # gate and up side by side in the rows of one tensor
            gu = normal(T, 2 * f).to(dt)
            g, u = gu[:, :f], gu[:, f:]
        else:
            g, u = normal(T, f).to(dt), normal(T, f).to(dt)
        return dict(g=g, u=u, dh=normal(T, f, scale=1e-2).to(dt))
    # balance: logits of a router that favours some experts, the ids it chose,
    # the combine weights of those and their gradients from the experts' outputs
    T, ne, k = case["T"], case["E"], case["k"]
    logits = (normal(T, ne) + normal(ne)).to(dt)
    chosen, ids = torch.topk(logits.float(), k, dim=1)
    w = torch.softmax(chosen, 1)
    if case["rule"] != "softmax":
        w = torch.sigmoid(chosen)
        if case["rule"] == "sigmoid_norm":
            w = w / w.sum(1, keepdim=True)
    ids = ids.to(torch.int32)
    if case["dropped"]:
        ids = torch.where(torch.rand(T, k, generator=gen, device="cuda") < case["dropped"],
                          torch.full_like(ids, -1), ids)
    mask = None
    if case["masked"]:
        mask = (torch.rand(T, generator=gen, device="cuda") >= case["masked"]).to(torch.uint8)
    s = dict(logits=logits, ids=ids, mask=mask, dloss=torch.full((1,), 1.0, device="cuda"), w=None, dw=None)
    if case["weights"]:
        s.update(w=w.contiguous(), dw=normal(T, k, scale=1e-2))
    return s


ALPHA = 0.01  # weight of the balance loss


def prepare(case, seed):
    st = dict(case=case, own=own, **_inputs(case, seed))
    if not own:
        return st
    from mxfp4_routed_expert_select_gb300 import k3moe as k
    st["k"] = k
    dt, op = _DT[case["dtype"]], case["op"]

    def new(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "quantise":
        r, c = case["rows"], case["cols"]
        if case["along"] != "cols":
            st.update(row=k.MxOperand(r, c), vrow=new(r, c))
        if case["along"] != "rows":
            st.update(col=k.MxOperand(c, r), vcol=new(c, r))
    elif op == "product":
        st.update(qx=k.MxOperand(case["M"], case["K"]), y=new(case["M"], case["N"]),
                  qw=k.MxOperand.from_matrix(st["packed"], st["scales"], case["N"], case["K"]))
    elif op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        st.update(xr=k.MxOperand(T, K), xc=k.MxOperand(K, T), wr=k.MxOperand(N, K), wc=k.MxOperand(K, N),
                  gr=k.MxOperand(T, N), gc=k.MxOperand(N, T), y=new(T, N), dx=new(T, K),
                  dw=new(N, K, dtype=torch.float32))
    elif op == "swiglu":
        T, f = case["T"], case["f"]
        st.update(h=new(T, f), ckpt=k.SwigluCheckpoint(T, f))
        if case["fused"]:
            st["dgu"] = new(T, 2 * f)
            st["dg"], st["du"] = st["dgu"][:, :f], st["dgu"][:, f:]
        else:
            st.update(dg=new(T, f), du=new(T, f))
    else:
        st.update(bal=k.BalanceLoss(case["E"], case["k"], ALPHA, case["rule"]), loss=new(1, dtype=torch.float32),
                  counts=new(case["E"], dtype=torch.int32), valid=new(1, dtype=torch.int32),
                  dlogits=new(case["T"], case["E"]))
    return st


# ----------------------------------------------------------- the plain forms

def _pow2(e):
    """2^e of whole numbers, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx(x):
    """The MXFP4 values of x along its last axis (32 to a block)."""
    x = x.float()
    k = x.shape[-1]
    v = torch.nn.functional.pad(x, (0, -k % 32)).unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(min=-127)  # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = v.abs().double() * _pow2(-e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0) * _pow2(e)
    return torch.copysign(q, v.double()).float().flatten(-2)[..., :k]


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _stored(packed, scales, k):
    """The values of a stored MXFP4 matrix."""
    lut = torch.tensor(_E2M1, device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(1).long()
    v = lut[codes].unflatten(1, (-1, 32)) * _pow2(scales.long() - 127).float().unsqueeze(-1)
    return v.flatten(1)[:, :k]


def _e4m3(x):
    """x as e4m3 values with one power-of-two scale per 32 along the rows."""
    x = x.float()
    k = x.shape[1]
    v = torch.nn.functional.pad(x, (0, -k % 32)).unflatten(1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    e = (e - 9 + (m > 0.875)).clamp(min=-127)  # the smallest with amax 2^-e <= 448
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = v.double() * _pow2(-e)
    step = _pow2((torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(a / step) * step * _pow2(e)).float().flatten(1)[:, :k]


def _plain_swiglu(s):
    dt = s["g"].dtype
    g, u = s["g"].float(), s["u"].float()
    h = (g / (1 + torch.exp(-g)) * u).to(dt)
    g, u, dh = _e4m3(s["g"]), _e4m3(s["u"]), s["dh"].float()
    sg = 1 / (1 + torch.exp(-g))
    dg = (dh * u * sg * (1 + g * (1 - sg))).to(dt)
    du = (dh * g * sg).to(dt)
    return (h, torch.cat((dg, du), 1)) if s["case"]["fused"] else (h, dg, du)


def _plain_balance(s):
    case = s["case"]
    l, ids, ne, k = s["logits"].float(), s["ids"].long(), case["E"], case["k"]
    on = torch.isfinite(l).any(1)
    if s["mask"] is not None:
        on = on & (s["mask"] != 0)
    n = on.sum()
    slot = on[:, None] & (ids >= 0) & (ids < ne)
    counts = torch.zeros(ne + 1, dtype=torch.int64, device=l.device)
    counts.index_add_(0, torch.where(slot, ids, torch.full_like(ids, ne)).flatten(),
                      torch.ones(ids.numel(), dtype=torch.int64, device=l.device))
    counts = counts[:ne]
    den = (k * n).clamp(min=1)
    if case["rule"] == "softmax":
        x = torch.exp(l - l.amax(1, keepdim=True))
    else:
        x = 1 / (1 + torch.exp(-l))
    tot = x.sum(1, keepdim=True)
    p = torch.where(on[:, None], x / tot, torch.zeros_like(x))
    f1 = ((ne * counts - den).double() / den.double())  # f - 1, which is what the gradient sees
    pm = p.double().sum(0) / n.clamp(min=1)
    loss = ALPHA * ((f1 + 1) * pm).sum() * (n > 0)
    f1 = f1.float()
    gl = ALPHA * s["dloss"] / n.clamp(min=1) * (f1 - (f1 * p).sum(1, keepdim=True))
    if case["rule"] == "softmax":
        d = p * gl
    else:
        d = p * (1 - x) * gl
    d = torch.where(on[:, None], d, torch.zeros_like(d))
    if s["dw"] is not None:
        w, dw = s["w"], s["dw"]
        w = torch.where(slot, w, torch.zeros_like(w))
        inner = (w * dw).sum(1, keepdim=True)
        at = torch.where(slot, ids, torch.zeros_like(ids))
        if case["rule"] == "softmax":
            c = w * (dw - inner)
        else:
            sc = torch.gather(x, 1, at)
            c = sc * (1 - sc) * dw if case["rule"] == "sigmoid" else w * (1 - sc) * (dw - inner)
        d = d.scatter_add(1, at, torch.where(slot, c, torch.zeros_like(c)))
    return (loss.float().reshape(1), counts.to(torch.int32), n.to(torch.int32).reshape(1), d.to(s["logits"].dtype))


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantise":
        out = []
        if case["along"] != "cols":
            out.append(_mx(s["x"]).to(s["x"].dtype))
        if case["along"] != "rows":
            out.append(_mx(s["x"].t().contiguous()).to(s["x"].dtype))
        return tuple(out)
    if op == "product":
        return (_mx(s["x"]) @ _stored(s["packed"], s["scales"], case["K"]).t()).to(s["x"].dtype)
    if op == "linear":
        x, w, dy, dt = s["x"], s["w"], s["dy"], s["x"].dtype
        y = _mx(x) @ _mx(w).t()
        dx = _mx(dy) @ _mx(w.t().contiguous()).t()
        dw = _mx(dy.t().contiguous()) @ _mx(x.t().contiguous()).t()
        return y.to(dt), dx.to(dt), dw
    return _plain_swiglu(s) if op == "swiglu" else _plain_balance(s)


# --------------------------------------------------------- the library's calls

def run(s):
    if not s["own"]:
        return _plain(s)
    k, op = s["k"], s["case"]["op"]
    if op == "quantise":
        row, col = s.get("row"), s.get("col")
        k.mx_quantize_operand(s["x"], row, col)
        out = []
        if row is not None:
            k.mx_dequantize(s["vrow"], row)
            out.append(s["vrow"])
        if col is not None:
            k.mx_dequantize(s["vcol"], col)
            out.append(s["vcol"])
        return tuple(out)
    if op == "product":
        k.mx_quantize_operand(s["x"], s["qx"])
        k.mx_matmul(s["y"], s["qx"], s["qw"])
        return s["y"]
    if op == "linear":
        k.mx_quantize_operand(s["x"], s["xr"], s["xc"])
        k.mx_quantize_operand(s["w"], s["wr"], s["wc"])
        k.mx_matmul(s["y"], s["xr"], s["wr"])
        k.mx_quantize_operand(s["dy"], s["gr"], s["gc"])
        k.mx_matmul(s["dx"], s["gr"], s["wc"])
        k.mx_matmul(s["dw"], s["gc"], s["xc"])
        return s["y"], s["dx"], s["dw"]
    if op == "swiglu":
        k.swiglu_forward(s["h"], s["ckpt"], s["g"], s["u"])
        k.swiglu_backward(s["dg"], s["du"], s["dh"], s["ckpt"])
        return (s["h"], s["dgu"]) if s["case"]["fused"] else (s["h"], s["dg"], s["du"])
    b = s["bal"]
    b.forward(s["loss"], s["counts"], s["valid"], s["logits"], s["ids"], s["mask"])
    b.backward(s["dlogits"], s["logits"], s["ids"], s["counts"], s["valid"], s["dloss"], s["mask"], s["w"], s["dw"])
    return s["loss"], s["counts"], s["valid"], s["dlogits"]


def work(case):
    es, op = (4 if case["dtype"] == "f32" else 2), case["op"]
    mx = 17 / 32  # bytes of an MXFP4 value
    if op == "quantise":
        n, sides = case["rows"] * case["cols"], 2 if case["along"] == "both" else 1
        return dict(bytes=n * es + sides * n * (mx + es), flops=4 * n * sides)
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=M * K * es + N * K * mx + M * N * es, flops=2 * M * N * K)
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        return dict(bytes=2 * es * (T * K + T * N) + N * K * (es + 4), flops=6 * T * N * K)
    if op == "swiglu":
        n = case["T"] * case["f"]
        return dict(bytes=n * es * 6, flops=20 * n)
    n, slots = case["T"] * case["E"], case["T"] * case["k"]
    return dict(bytes=2 * n * es + 4 * slots * (3 if case["weights"] else 1), flops=12 * n)


# ---------------------------------------------- the definitions in 64 bits

def _two(e):
    """2^e of whole numbers from -300 to 300, looked up."""
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=e.device)[e.long() + 300]


def _mx64(x):
    """Each value to the nearest of the eight magnitudes by its thresholds
    (the halfway points, which go to the even code)."""
    x = x.double()
    k = x.shape[1]
    n = -(-k // 32) * 32
    v = torch.zeros(x.shape[0], n, dtype=torch.float64, device=x.device)
    v[:, :k] = x
    v = v.view(x.shape[0], n // 32, 32)
    top = v.abs().max(-1, keepdim=True).values
    e = torch.round(torch.log2(top.clamp(min=2.0 ** -149)))
    e = torch.where(_two(e) > top, e - 1, e) - 2
    scale = _two(e.clamp(min=-127))
    a = v.abs() / scale
    code = torch.zeros(a.shape, dtype=torch.int64, device=x.device)
    for i, (edge, up) in enumerate([(.25, False), (.75, True), (1.25, False), (1.75, True), (2.5, False),
                                    (3.5, True), (5.0, False)]):
        code += (a >= edge) if up else (a > edge)
    mag = torch.tensor(_E2M1[:8], dtype=torch.float64, device=x.device)[code]
    return (torch.where(torch.signbit(v), -mag, mag) * scale).view(x.shape[0], n)[:, :k]


def _e4m3_64(x):
    """Each value to the nearest entry of the e4m3 table, ties to the even one."""
    x = x.double()
    T, k = x.shape
    n = -(-k // 32) * 32
    v = torch.zeros(T, n, dtype=torch.float64, device=x.device)
    v[:, :k] = x
    v = v.view(T, n // 32, 32)
    top = v.abs().max(-1, keepdim=True).values
    s = _two(torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -127))))
    s = torch.where(top / s > 448, 2 * s, torch.where(top / (s / 2) <= 448, s / 2, s)).clamp(min=2.0 ** -127)
    table = [i * 2.0 ** -9 for i in range(8)] + [(8 + m) * 2.0 ** (p - 3) for p in range(-6, 9) for m in range(8)]
    table = torch.tensor(table[:127], dtype=torch.float64, device=x.device)
    mids = (table[1:] + table[:-1]) / 2
    a = v.abs() / s
    i = torch.searchsorted(mids, a)
    j = i.clamp(max=mids.numel() - 1)
    i = torch.where((i < mids.numel()) & (mids[j] == a) & (i % 2 == 1), i + 1, i)
    return (torch.where(v < 0, -table[i], table[i]) * s).view(T, n)[:, :k]


def _exact_balance(case, s):
    l, ids, ne, k = s["logits"].double(), s["ids"].long(), case["E"], case["k"]
    keep = (l > float("-inf")).any(1)
    if s["mask"] is not None:
        keep &= s["mask"].bool()
    n = int(keep.sum())
    hit = torch.nn.functional.one_hot(ids.clamp(min=0), ne) * (ids >= 0).unsqueeze(-1) if ids.numel() < 2 ** 14 else None
    if hit is None:
        hit = torch.zeros(l.shape, dtype=torch.int64, device=l.device)
        for j in range(k):
            ok = (ids[:, j] >= 0).nonzero().flatten()
            hit[ok, ids[ok, j]] += 1
    else:
        hit = hit.sum(1)
    counts = (hit * keep.unsqueeze(1)).sum(0)
    d = torch.zeros_like(l)
    if n == 0:
        return torch.zeros(1, dtype=torch.float64, device=l.device), counts, n, d
    f = counts.double() * ne / (k * n)
    sg = torch.sigmoid(l)
    p = torch.softmax(l, 1) if case["rule"] == "softmax" else sg / sg.sum(1, keepdim=True)
    p, r = p[keep], sg[keep]
    loss = ALPHA * (f * p.mean(0)).sum()
    d[keep] = ALPHA * float(s["dloss"]) / n * p * (f - (p @ f).unsqueeze(1)) * (1 if case["rule"] == "softmax" else 1 - r)
    if s["dw"] is not None:
        for j in range(k):
            row = (keep & (ids[:, j] >= 0)).nonzero().flatten()
            col = ids[row, j]
            w, dw = s["w"].double(), s["dw"].double()
            dot = (w * dw * (ids >= 0)).sum(1)[row]
            w, dw, q = w[row, j], dw[row, j], sg[row, col]
            if case["rule"] == "softmax":
                d[row, col] += w * (dw - dot)
            elif case["rule"] == "sigmoid":
                d[row, col] += dw * q * (1 - q)
            else:
                d[row, col] += w * (dw - dot) * (1 - q)
    return loss.reshape(1), counts, n, d


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op == "quantise":
        x, along = s["x"], case["along"]
        return tuple(([_mx64(x)] if along != "cols" else []) + ([_mx64(x.t())] if along != "rows" else []))
    if op == "product":
        mag = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
        w = torch.empty(case["N"], s["packed"].shape[1] * 2, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = mag[(s["packed"] % 16).long()], mag[(s["packed"] // 16).long()]
        w *= _two(s["scales"].long() - 127).repeat_interleave(32, 1)
        return _mx64(s["x"]) @ w[:, :case["K"]].t()
    if op == "linear":
        x, w, dy = s["x"], s["w"], s["dy"]
        return (_mx64(x) @ _mx64(w).t(), _mx64(dy) @ _mx64(w.t()).t(), _mx64(dy.t()) @ _mx64(x.t()).t())
    if op == "swiglu":
        g, u = s["g"].double(), s["u"].double()
        h = g * torch.sigmoid(g) * u
        g, u, dh = _e4m3_64(s["g"]), _e4m3_64(s["u"]), s["dh"].double()
        r = torch.sigmoid(g)
        dg, du = dh * u * (r + g * r * (1 - r)), dh * g * r
        return (h, torch.cat((dg, du), 1)) if case["fused"] else (h, dg, du)
    loss, counts, n, d = _exact_balance(case, s)
    return loss, counts.to(torch.int32), torch.tensor([n], dtype=torch.int32, device="cuda"), d
