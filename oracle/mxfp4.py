"""Microscaled 4-bit floating point in 64 bits: quantiser, values, products.

e2m1 elements, one scale 2^(c - 127) per 32 elements of a row; c the least code
with 6 * 2^(c - 127) >= amax, clamped to [0, 253]; 127 for a block of zeros;
255 (NaN), with zero elements, for a block with a NaN or an infinity.
"""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quant_mxfp4(x):
    """x [..., rows, K] fp32 -> (codes uint8 [..., rows, K/2], words int32 [..., K/128, rows])."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    v = np.where(bad[..., None], 0.0, b)
    amax = np.abs(v).max(-1)
    c = np.full(amax.shape, 127, dtype=np.int64)
    nz = amax > 0
    m, e = np.frexp(amax[nz])  # amax = m 2^e, m in [0.5, 1); 6 * 2^s = 0.75 * 2^(s + 3)
    c[nz] = np.clip(np.where(m <= 0.75, e - 3, e - 2) + 127, 0, 253)
    y = np.abs(v) * 2.0 ** (127.0 - c)[..., None]
    # nearest grid value; of two equally near ones the even code
    d = np.abs(y[..., None] - E2M1)
    near = d.min(-1, keepdims=True)
    cand = d == near
    odd = np.arange(8) % 2
    code = np.argmax(np.where(cand, 2 - odd, 0), -1)
    code = np.where(bad[..., None], 0, code | np.where(np.signbit(b), 8, 0)).astype(np.uint8)
    code = code.reshape(x.shape[:-1] + (-1, 2))
    c = np.where(bad, 255, c).astype(np.uint8)
    return code[..., 0] | (code[..., 1] << 4), pack_words(c)


def pack_words(c):
    """Scale codes [..., rows, K/32] -> words [..., K/128, rows], block 4 w + j in byte j."""
    c = np.asarray(c).astype(np.uint32).reshape(c.shape[:-1] + (-1, 4))
    w = c[..., 0] | c[..., 1] << 8 | c[..., 2] << 16 | c[..., 3] << 24
    return np.ascontiguousarray(np.swapaxes(w, -1, -2)).view(np.int32)


def unpack_words(w):
    u = np.swapaxes(np.ascontiguousarray(w).view(np.uint32), -1, -2)
    c = np.stack([(u >> (8 * j)) & 255 for j in range(4)], -1)
    return c.reshape(u.shape[:-1] + (-1,))


def values_mxfp4(codes, words):
    """The elements' values in fp64."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.int64)
    v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    c = unpack_words(words).astype(np.float64)
    s = np.where(c == 255, np.nan, 2.0 ** (c - 127))
    return (v.reshape(v.shape[:-1] + (-1, 32)) * s[..., None]).reshape(v.shape)


def gemm_mxfp4(a, sfa, b, sfb):
    """(A . B^T, sum of |a| |b|) in fp64."""
    va, vb = values_mxfp4(a, sfa), values_mxfp4(b, sfb)
    return va @ vb.T, np.abs(va) @ np.abs(vb).T
