"""Dense 8-bit operators around the layer in fp64: RMS norm with the residual
addition, int8 and e4m3 row quantization, the int8 product with a scale per
token and channel, the e4m3 product with a scale per block of 128, and their
gated forms.

The pages name none of these; the readings are the header's: y = v * r * w with
v = x + res and r = 1 / sqrt(mean(v^2) + eps); int8 codes round(y * 127 / m)
with m = max(max|y|, 2^-100) and scale m / 127; sums of int8 products are
exact integers (held in fp64, exact below 2^53).
"""
import numpy as np

from .numerics import e4m3_decode

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


def fp8_values(codes, block_scales):
    """e4m3 codes [rows, K] times a scale per 128 columns [rows, ceil(K / 128)], fp64."""
    rows, K = codes.shape
    wide = np.repeat(np.asarray(block_scales, dtype=np.float64), 128, axis=1)[:, :K]
    return e4m3_decode(codes) * wide


def e8m0(b):
    """E8M0 bytes as fp64: 2^(b - 127), 255 is NaN."""
    b = np.asarray(b).astype(np.float64)
    return np.where(b == 255, np.nan, np.exp2(b - 127))


def weight_values(codes, sb):
    """e4m3 codes [N, K] with an fp32 scale per 128 x 128 block, fp64."""
    per_row = np.repeat(np.asarray(sb, dtype=np.float64), 128, axis=0)[:codes.shape[0]]
    return fp8_values(codes, per_row)


def gemm_fp8(a, sa, b, sb, bias=None, add=None):
    """Returns (sum of the terms' magnitudes, out), both unrounded fp64."""
    va, vb = fp8_values(a, e8m0(sa)), weight_values(b, sb)
    out, mag = va @ vb.T, np.abs(va) @ np.abs(vb).T
    if bias is not None:
        out = out + np.asarray(bias, dtype=np.float64)[None, :]
        mag = mag + np.abs(np.asarray(bias, dtype=np.float64))[None, :]
    if add is not None:
        out = out + np.asarray(add, dtype=np.float64)
        mag = mag + np.abs(np.asarray(add, dtype=np.float64))
    return mag, out


def glu_fp8(a, sa, w13, s13):
    """Returns (g, u, magnitudes of g, of u, h): h = silu(g) * u."""
    inter, half = w13.shape[0] // 2, s13.shape[0] // 2
    mg, g = gemm_fp8(a, sa, w13[:inter], s13[:half])
    mu, u = gemm_fp8(a, sa, w13[inter:], s13[half:])
    e = np.exp(-np.abs(g))
    sig = np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
    return g, u, mg, mu, g * sig * u


def fp8_largest(a, sa, b, sb):
    """Per output, the largest product of |a| and |b| that each block of 128 could hold, scaled and summed over the blocks."""
    K = a.shape[1]
    kb = (K + 127) // 128

    def tops(codes):
        v = np.zeros((codes.shape[0], kb * 128))
        v[:, :K] = np.abs(e4m3_decode(codes))
        return v.reshape(codes.shape[0], kb, 128).max(axis=2)
    return (tops(a) * e8m0(sa)) @ (tops(b) * np.abs(np.repeat(np.asarray(sb, dtype=np.float64), 128, axis=0)[:b.shape[0]])).T
