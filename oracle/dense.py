"""Dense 8-bit operators around the layer in fp64: RMS norm with the residual
addition, int8 and e4m3 row quantization, the int8 product with a scale per
token and channel, and its gated form.

The pages name none of these; the readings are the header's: y = v * r * w with
v = x + res and r = 1 / sqrt(mean(v^2) + eps); int8 codes round(y * 127 / m)
with m = max(max|y|, 2^-100) and scale m / 127; sums of int8 products are
exact integers (held in fp64, exact below 2^53).
"""
import numpy as np

I8_FLOOR = 2.0 ** -100


def rms_norm(x, weight=None, eps=1e-6, res=None):
    """x, res: fp64 rows. Returns (y, v) unrounded."""
    v = np.asarray(x, dtype=np.float64)
    if res is not None:
        v = v + np.asarray(res, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    y = v * r
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)[None, :]
    return y, v


def i8_rows(y):
    """(codes before rounding, scales): codes are rint of the first."""
    m = np.maximum(np.abs(y).max(axis=1), I8_FLOOR)
    return y * (127.0 / m)[:, None], m / 127.0


def gemm_i8(a, sa, b, sb, bias=None, add=None):
    """Returns (product scaled, out), both unrounded fp64."""
    p = a.astype(np.float64) @ b.astype(np.float64).T
    p = p * np.asarray(sa, dtype=np.float64)[:, None] * np.asarray(sb, dtype=np.float64)[None, :]
    out = p
    if bias is not None:
        out = out + np.asarray(bias, dtype=np.float64)[None, :]
    if add is not None:
        out = out + np.asarray(add, dtype=np.float64)
    return p, out


def glu_i8(a, sa, w13, s13):
    """Returns (g, u, h): h = silu(g) * u."""
    p, _ = gemm_i8(a, sa, w13, s13)
    inter = w13.shape[0] // 2
    g, u = p[:, :inter], p[:, inter:]
    e = np.exp(-np.abs(g))
    sig = np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
    return g, u, g * sig * u
