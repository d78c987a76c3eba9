"""Calls that take longer than the limit of a wait, while each of their steps is short,
end with their results: a library built with limits of half a millisecond in the place
of two seconds runs calls of a few milliseconds.  Whole numbers below 2^24, so that every
sum is exact."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from mxfp4_routed_expert_select_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    return _build.build(force=True, extra=["-DK3_WAIT_LIMIT_NS=500000ull"],
                        so=str(tmp_path_factory.mktemp("limits") / "libk3moe.so"))


def _run(library, case):
    r = subprocess.run([sys.executable, __file__, case], env=dict(os.environ, K3MOE_LIBRARY=library), cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_weight_gradients_of_a_long_group(library):
    _run(library, "long_group")


def test_operands_of_a_long_sum(library):
    _run(library, "long_sum")


# Many short tiles: the second CTA of a pair waits for the end of the call only when that
# is near.
@pytest.mark.parametrize("case", ["many_grouped_tiles", "many_gradient_tiles", "many_operand_tiles"])
def test_pairs_with_many_tiles(library, case):
    _run(library, case)


# ---------------------------------------------------- what the library's process runs

def _whole(gen, *shape):
    return torch.randint(-1, 2, shape, generator=gen, device="cuda", dtype=torch.int8).bfloat16()


def _timed(k, call):
    """Milliseconds of the second of two calls; no wait of either has run out."""
    call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    call()
    b.record()
    torch.cuda.synchronize()
    assert k.device_error() == 0
    ms = a.elapsed_time(b)
    assert ms > 1, "the call took %.2f ms, no longer than a wait may" % ms


def long_group(k, gen):
    """One tile whose sum runs over 2^21 rows."""
    rows = 1 << 21
    groups = k.ExpertGroups(1, 1, rows)
    groups.plan(torch.zeros(rows, 1, dtype=torch.int32, device="cuda"))
    dy, x, dw = _whole(gen, rows, 8), _whole(gen, rows, 8), torch.full((1, 8, 8), 0.5, device="cuda")
    _timed(k, lambda: k.grouped_wgrad(dw, dy, x, groups))
    assert torch.equal(dw[0].double(), dy.double().t() @ x.double())


def long_sum(k, gen):
    """Tiles of 2^25 columns, shared by eight CTAs: codes of 0, 1 and -1."""
    rows, K = 16, 1 << 25
    ops, values = [], []
    for _ in range(2):
        v = torch.randint(-1, 2, (rows, K), generator=gen, device="cuda", dtype=torch.int8)
        c = (v == 1) * 2 + (v == -1) * 10  # E2M1: 1.0 is code 2, the sign bit 3
        op = k.MxOperand(rows, K)
        op.codes.copy_((c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8).flatten())
        op.atoms.fill_(127)
        ops.append(op)
        values.append(v)
    C = torch.full((rows, rows), 0.5, device="cuda")
    _timed(k, lambda: k.mx_matmul(C, *ops))
    want = sum(a.double() @ b.double().t() for a, b in zip(*(v.split(1 << 22, 1) for v in values)))
    assert torch.equal(C.double(), want)


def _slots(k, gen, E, top_k, T):
    """A plan of T tokens, and the ids grouped."""
    ids = torch.randint(0, E, (T, top_k), generator=gen, device="cuda", dtype=torch.int32)
    groups = k.ExpertGroups(E, top_k, T)
    groups.plan(ids)
    return groups


def many_grouped_tiles(k, gen):
    E, top_k, T, N, K = 4, 2, 1 << 17, 2048, 4096
    groups = _slots(k, gen, E, top_k, T)
    assert k.grouped_matmul_form(E, T * top_k, N, K) == 256
    packed = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8) & 0x22  # 0 and 1
    W = k.MxExperts.from_matrices(packed, torch.full((E, N, K // 32), 127, device="cuda", dtype=torch.uint8))
    x, a = _whole(gen, T, K), k.Mx8Rows(T, K)
    k.mx8_quantize(a, x)
    C = torch.full((T * top_k, N), 0.5, device="cuda")
    _timed(k, lambda: k.grouped_matmul(C, a, W, groups, gather=True))
    off = groups.offsets.tolist()
    V = torch.stack(((packed & 15) // 2, (packed >> 4) // 2), -1).flatten(-2).bfloat16()
    for e in range(E):
        for s in (slice(off[e], off[e] + 300), slice(off[e + 1] - 300, off[e + 1])):
            assert torch.equal(C[s].double(), x[groups.order[s].long() // top_k].double() @ V[e].double().t())


def many_gradient_tiles(k, gen):
    E, top_k, T, N, K = 16, 4, 1 << 17, 2048, 2048
    groups = _slots(k, gen, E, top_k, T)
    dy, x, dw = _whole(gen, T * top_k, N), _whole(gen, T, K), torch.full((E, N, K), 0.5, device="cuda")
    _timed(k, lambda: k.grouped_wgrad(dw, dy, x, groups, gather=True))
    off = groups.offsets.tolist()
    for e in (0, E - 1):
        s = slice(off[e], off[e + 1])
        assert torch.equal(dw[e].double(), dy[s].double().t() @ x[groups.order[s].long() // top_k].double())


def many_operand_tiles(k, gen):
    M, N, K = 32768, 16384, 16384
    ops, values = [], []
    for rows in (M, N):
        v = _whole(gen, rows, K)
        v[:, ::32] = 1  # every block's largest is 1: kept exactly
        op = k.MxOperand(rows, K)
        k.mx_quantize_operand(v, op)
        ops.append(op)
        values.append(v)
    C = torch.full((M, N), 0.5, device="cuda")
    assert k.mx_matmul_form(M, N, K, C.dtype)[0]
    _timed(k, lambda: k.mx_matmul(C, *ops))
    for s in (slice(0, 256), slice(M - 256, M)):
        assert torch.equal(C[s].double(), values[0][s].double() @ values[1].double().t())


if __name__ == "__main__":
    sys.path.insert(0, ROOT)
    from mxfp4_routed_expert_select_gb300 import k3moe
    globals()[sys.argv[1]](k3moe, torch.Generator(device="cuda").manual_seed(1))
