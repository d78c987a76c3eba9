"""Plain 64-bit forms of the MXFP4 operands, used by the tests of the operand
calls: the block conversion through the oracle, the operand's scale atoms read
back by their definition, and the values a set of codes and bytes stands for."""
import numpy as np

import oracle


def quantize(x):
    """(codes [rows][ceil32(in)], bytes [rows][ceil32(in)/32]) of x by the oracle."""
    x = np.asarray(x, np.float32)
    rows, n = x.shape
    pad = -(-n // 32) * 32
    v = np.zeros((rows, pad), np.float32)
    v[:, :n] = x
    _, codes, scales = oracle.mx_quantize(v)
    return codes.reshape(rows, pad), scales.reshape(rows, pad // 32)


def unpack(packed):
    packed = np.asarray(packed)
    c = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    c[:, 0::2] = packed & 15
    c[:, 1::2] = packed >> 4
    return c


MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def values(codes, scales):
    """The fp64 values; byte 255 is NaN."""
    v = np.where(codes & 8, -1.0, 1.0) * MAG[codes & 7]
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s[scales == 255] = np.nan
    return v * np.repeat(s, 32, axis=1)


def atoms_to_scales(atoms, rows, n):
    """Scale bytes [rows][ceil32(n)/32] out of an operand's atoms, and whether
    every byte past the matrix is zero."""
    nk = 2 * -(-n // 256)
    a = np.asarray(atoms).reshape(-(-rows // 128), nk, 32, 4, 4)  # row tile, k atom, r % 32, r / 32, block
    full = a.transpose(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, nk * 4)
    nb = -(-n // 32)
    rest = full.copy()
    rest[:rows, :nb] = 0
    return full[:rows, :nb], not rest.any()
