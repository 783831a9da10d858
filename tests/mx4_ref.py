"""Plain 64-bit forms of the norm and of rows in 4-bit blocks (include/sparse_ffn_mx4.h) in numpy,
for the tests. They share nothing with the library."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(x):
    """Rows of numbers -> codes 0..15 [R, B, 32] and scale bytes [R, B]: the scale by search over
    all of them, each code by its distances to the whole grid."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    B = (K + 31) // 32
    v = np.zeros((R, B * 32))
    v[:, :K] = x
    v = v.reshape(R, B, 32)
    m = np.abs(v).max(axis=2)
    with np.errstate(invalid="ignore", over="ignore"):
        bad = ~np.isfinite(m)
        # the smallest E from 0 on whose 7 * 2^(E - 127) is above m
        E = np.searchsorted(7.0 * 2.0 ** (np.arange(255) - 127.0), np.where(bad, 0.0, m), side="right")
        t = np.abs(np.where(bad[:, :, None], 0.0, v)) / (2.0 ** (E - 127.0))[:, :, None]
    far = np.abs(t[..., None] - GRID)
    near = far.min(axis=3, keepdims=True)
    # of two codes equally near the even one
    even = np.arange(8) % 2 == 0
    code = np.where((far == near) & even, 2, np.where(far == near, 1, 0)).argmax(axis=3)
    code = code + 8 * np.signbit(v)
    code[bad] = 0
    return code, np.where(bad, 255, E)


def pack(code, E):
    """Codes and scale bytes as the library lays them out, without room behind the scales."""
    code = code.reshape(code.shape[0], -1, 2).astype(np.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), E.astype(np.uint8)


def values(q, E):
    """The values of packed rows."""
    q = np.asarray(q)
    c = np.stack((q & 15, q >> 4), axis=2).reshape(q.shape[0], -1)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(np.asarray(E) == 255, np.nan, 2.0 ** (np.asarray(E, np.float64) - 127.0))
    return (v.reshape(q.shape[0], -1, 32) * s[:, :, None]).reshape(q.shape[0], -1)


def matmul(x, w, bias=None):
    """(y, magnitude): y in 64 bits of rows of values, and the sum of |products| and |bias|."""
    b = 0.0 if bias is None else np.asarray(bias, np.float64)
    with np.errstate(invalid="ignore"):
        return x @ w.T + b, np.abs(x) @ np.abs(w).T + np.abs(b)


def norm(v, w=None, eps=1e-6):
    """Rows v (the residual already added) in 64 bits."""
    v = np.asarray(v, np.float64)
    w = 1.0 if w is None else np.asarray(w, np.float64)
    with np.errstate(all="ignore"):
        return v * w / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
