"""Plain 64-bit forms for the tests of the 8-bit rows and of what is grouped by
expert: the block conversion to e4m3 by the table, rows read back by their layout,
and the plan of a routed batch."""
import numpy as np

TABLE = np.array([m * 2.0 ** -9 for m in range(8)] +
                 [(8 + m) * 2.0 ** (p - 3) for p in range(-6, 9) for m in range(8)][:119])  # 0 .. 448


def quantize(x):
    """(values [T][n], scale bytes [T][ceil32(n)/32]) of fp32 rows."""
    x = np.asarray(x, np.float32).astype(np.float64)
    T, n = x.shape
    pad = -(-n // 32) * 32
    v = np.zeros((T, pad))
    v[:, :n] = x
    v = v.reshape(T, pad // 32, 32)
    finite = np.isfinite(v).all(-1)
    top = np.abs(np.where(finite[..., None], v, 0.0)).max(-1)
    m, e = np.frexp(top)  # top = m 2^e, .5 <= m < 1; 448 = .875 * 2^9
    e = np.where(top > 0, e - 9 + (m > 0.875) + 127, 0).clip(0)
    a = np.abs(np.where(finite[..., None], v, 0.0)) * np.ldexp(1.0, 127 - e)[..., None]
    lo = np.clip(np.searchsorted(TABLE, a, side="right") - 1, 0, TABLE.size - 1)
    hi = np.minimum(lo + 1, TABLE.size - 1)
    d = (a - TABLE[lo]) - (TABLE[hi] - a)
    up = (d > 0) | ((d == 0) & (lo % 2 == 1))
    q = TABLE[np.where(up & (hi > lo), hi, lo)] * np.ldexp(1.0, e - 127)[..., None]
    q = np.minimum(np.where(np.signbit(v), -q, q), 240 * 2.0 ** 120).clip(-240 * 2.0 ** 120)
    q[~finite] = np.nan
    return q.reshape(T, pad)[:, :n], np.where(finite, e, 255)


def read_rows(rows8):
    """(values [T][n], scale bytes [T][ceil32(n)/32], whether all past n is zero) of a
    k3moe.Mx8Rows."""
    T, n = rows8.rows, rows8.in_
    pad, nb = -(-n // 32) * 32, -(-n // 32)
    c = rows8.codes.cpu().numpy().reshape(T, pad)
    s = rows8.scales.cpu().numpy().reshape(T, 4 * -(-n // 128))
    clean = not c[:, n:].any() and not s[:, nb:].any()
    s = s[:, :nb].astype(np.int64)
    scale = np.ldexp(1.0, s - 127)
    scale[s == 255] = np.nan
    v = np.where(c & 128, -1.0, 1.0) * TABLE[np.minimum(c & 127, 126)] * np.repeat(scale, 32, axis=1)
    return v[:, :n], s, clean


def plan(ids, E):
    """(offsets, order, pos) of ids [T][k]."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    flat = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[order], np.arange(E + 1))
    pos = np.empty_like(order)
    pos[order] = np.arange(flat.size)
    kept = offsets[E]
    pos[flat == E] = -1
    order = order.copy()
    order[kept:] = -1
    return offsets, order, pos
