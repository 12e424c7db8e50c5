"""MXFP4 in float64: quantisation of rows and weights, and the W4A4 expert FFN.

Format (OCP microscaling; E2M1 codes, one E8M0 scale per 32 consecutive values):
e = floor(log2 max|x|) - 2, at least -127 (0 for a group of zeros), scale byte
e + 127; each value divided by 2^e goes to the nearest E2M1 magnitude, ties to
the even code, magnitudes past 6 to 6, the sign kept. A group that holds a NaN or
an infinity has scale byte 255 and codes 0."""
from __future__ import annotations

import numpy as np

from .ref import dequant_mxfp4, e2m1_decode, e8m0_decode

GROUP = 32
MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize_rows(x):
    """(codes [R, C/2], scale bytes [R, C/32]) of rows x [R, C]; byte i of a row
    holds columns 2i (low nibble) and 2i + 1."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    v = x.reshape(R, C // GROUP, GROUP)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    amax = np.abs(v).max(axis=2)
    _, ex = np.frexp(amax)                       # amax = m 2^ex, m in [1/2, 1): floor(log2) = ex - 1
    e = np.where(amax > 0, np.maximum(ex - 3, -127), 0)
    a = np.abs(np.ldexp(v, -e[:, :, None]))
    # the places of the borders between neighbouring magnitudes; the tie at a border
    # goes to the even one of the two codes
    code = np.zeros(a.shape, dtype=np.int64)
    for i in range(7):
        border = (MAGS[i] + MAGS[i + 1]) / 2
        code += (a >= border) if i % 2 else (a > border)
    code |= np.where(np.signbit(v), 8, 0)
    code = np.where(bad[:, :, None], 0, code).reshape(R, C).astype(np.uint8)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def row_values(q, s):
    """The values [R, C] that quantize_rows' codes and scales stand for."""
    q = np.asarray(q, dtype=np.uint8)
    v = np.empty((q.shape[0], 2 * q.shape[1]))
    v[:, 0::2], v[:, 1::2] = e2m1_decode(q & 15), e2m1_decode(q >> 4)
    return v * np.repeat(e8m0_decode(s), GROUP, axis=1)


def quantize_weights(w):
    """(codes [K/2, N], scale bytes [K/32, N]) of a matrix w [K, N], grouped along K."""
    q, s = quantize_rows(np.asarray(w, dtype=np.float64).T)
    return np.ascontiguousarray(q.T), np.ascontiguousarray(s.T)


def weight_values(q, s):
    return dequant_mxfp4(q, s)


def round_rows(x):
    return row_values(*quantize_rows(x))


def ffn(x, W1, W3, W2):
    """(y, g, u, h, hq) of one expert on its rows: x and the weights as the values
    their codes stand for; hq = h rounded to MXFP4."""
    g, u = x @ W1, x @ W3
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    hq = round_rows(h)
    return hq @ W2, g, u, h, hq
