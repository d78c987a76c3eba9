"""The norm's 8-bit rows against the codes of the 64-bit formula: only values within the
rounding of an fp32 y from a border between two codes may differ."""
import pytest
import torch

import e4m3_reference as ref
from mxfp4_routed_expert_select_gb300 import k3moe as k

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _pow2(e):
    """2^e of whole numbers, exactly (torch.ldexp forms it by a pow in fp32 on a GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _codes(y):
    """Values of fp64 rows in blocks of 32 as e4m3 with the smallest power of two s that has
    max / s <= 448, ties to even."""
    v = torch.nn.functional.pad(y, (0, -y.shape[1] % 32)).unflatten(1, (-1, 32))
    m, e = torch.frexp(v.abs().amax(-1, keepdim=True))  # max = m 2^e, .5 <= m < 1; 448 = .875 * 2^9
    s = _pow2(e - 9 + (m > 0.875))
    a = v / s
    step = _pow2((torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(a / step) * step * s).flatten(1)[:, :y.shape[1]]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,n,delta", [(1024, 7168, True), (1500, 4099, True), (300, 20000, False), (4000, 512, False)])
def test_codes_next_to_a_border(T, n, delta, dt):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (torch.randn(T, n, generator=g, device="cuda") * 3).to(DT[dt])
    d = torch.randn(T, n, generator=g, device="cuda").to(DT[dt]) if delta else None
    gain = 1 + torch.randn(n, generator=g, device="cuda") * 0.2
    y8 = k.Mx8Rows(T, n)
    k.RmsNorm(n, 1e-6).forward(None, x, d, gain=gain, y8=y8)
    r = (x.float() + d.float()).to(DT[dt]).double() if delta else x.double()
    eps = float(torch.tensor(1e-6, dtype=torch.float32))
    want = _codes(r / (r.square().mean(1, keepdim=True) + eps).sqrt() * gain.double())
    got, _, clean = ref.read_rows(y8)
    off = int((torch.from_numpy(got).cuda() != want).sum())
    # A code differs where a border lies between y and the exact value.  In a binade of eight
    # steps a value is twelve steps' eighths long on average, so an error of d times the value
    # passes a border in 12 d of them.  d: the two products 2 * 2^-24; the root half an ulp
    # and half of what the sum of squares is off, which is four roundings of 75 (they do not
    # all fall one way): 2 * 2^-24.  And one block whose largest value lies at 448.
    assert clean and off <= 12 * 4.6 * 2.0 ** -24 * T * n + 32, (off, T * n)
    print("%d x %d %s: %d of %d codes" % (T, n, dt, off, T * n))
