"""The int8 products give the same bits however their work is split: each row
and column of a product in every tile shape, on whole lines and on rows that
start anywhere, is what a product of those rows and columns alone gives.

The sum is an exact integer; what follows is, in this order, the conversion to
fp32, the row's scale, the column's scale with the bias in one rounding, the
addend: no step may depend on the tile. Signed zeros count.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from test_gpu_dense import _f32, _i8, _rng, _say

pytestmark = pytest.mark.gpu


def _same_bits(a, b):
    import torch
    t = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(t), b.contiguous().view(t))


# rows and columns of the whole product, and of parts of it that other tile shapes take
WHOLE = (4099, 1088)
PARTS = [(4099, 1088), (4099, 1000), (2500, 1087), (1024, 1088), (700, 513), (300, 1088), (200, 77), (64, 1088), (33, 64), (9, 1088), (1, 1088), (1, 5)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("bias,add", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("K", [144, 1024])
def test_products_do_not_depend_on_the_split(gpu, K, bias, add, f32):
    import torch
    M, N = WHOLE
    r = _rng(K, bias, add, f32, 71)
    a, b = r.integers(-128, 128, (M, K)), r.integers(-128, 128, (N, K))
    a[0], b[3] = 0, 0                                    # sums of zero ...
    sa, sb = 0.03 * np.exp(r.normal(size=M)), 0.03 * np.exp(r.normal(size=N))
    sa[::2] *= -1                                        # ... below zero: -0.0
    ot = torch.float32 if f32 else torch.bfloat16
    da, db, dsa, dsb = _i8(a, gpu), _i8(b, gpu), _f32(sa, gpu), _f32(sb, gpu)
    dbias = _f32(r.normal(size=N), gpu) if bias else None
    dadd = _f32(r.normal(size=(M, N)), gpu).to(ot) if add else None
    whole = moe.gemm_i8(da, dsa, db, dsb, bias=dbias, add=dadd, out_dtype=ot)
    for m, n in PARTS:
        part = moe.gemm_i8(da[:m], dsa[:m], db[:n], dsb[:n], bias=None if dbias is None else dbias[:n],
                           add=None if dadd is None else dadd[:m, :n].contiguous(), out_dtype=ot)
        torch.cuda.synchronize()
        d = (part != whole[:m, :n])
        _say(f"    {m} x {n}: {int(d.sum())} of {d.numel()} differ")
        assert _same_bits(part, whole[:m, :n]), (m, n)


@pytest.mark.parametrize("K", [144, 1024])
def test_gated_products_do_not_depend_on_the_split(gpu, K):
    import torch
    M, N = WHOLE
    r = _rng(K, 72)
    a, g, u = r.integers(-128, 128, (M, K)), r.integers(-128, 128, (N, K)), r.integers(-128, 128, (N, K))
    a[0], g[3] = 0, 0
    sa, sg, su = 0.03 * np.exp(r.normal(size=M)), 0.03 * np.exp(r.normal(size=N)), 0.03 * np.exp(r.normal(size=N))
    sa[::2] *= -1
    da, dsa = _i8(a, gpu), _f32(sa, gpu)
    whole = moe.glu_i8(da, dsa, _i8(np.concatenate([g, u]), gpu), _f32(np.concatenate([sg, su]), gpu))
    for m, n in PARTS:
        part = moe.glu_i8(da[:m], dsa[:m], _i8(np.concatenate([g[:n], u[:n]]), gpu), _f32(np.concatenate([sg[:n], su[:n]]), gpu))
        torch.cuda.synchronize()
        d = (part != whole[:m, :n])
        _say(f"    {m} x {n}: {int(d.sum())} of {d.numel()} differ")
        assert _same_bits(part, whole[:m, :n]), (m, n)
