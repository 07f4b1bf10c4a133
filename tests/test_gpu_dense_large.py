"""Dense operators where byte and element offsets pass 2^31 and 2^32.

The operands are too large for a 64-bit reference of all of them. Rows at the
start, at the end and on both sides of the offsets are checked: the products
against integers (sums are exact, scales are powers of two), the row operators
against the same call on those rows alone, which has to give the same bits
(fp64 sums of a row are taken in the same order whichever rows stand beside).
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from test_gpu_dense import _say

pytestmark = pytest.mark.gpu


def _codes(gpu, rows, cols, seed):
    """Random int8 codes, made on the device in pieces."""
    import torch
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    t = torch.empty(rows, cols, dtype=torch.int8, device=gpu)
    step = max(1, (1 << 28) // cols)
    for r in range(0, rows, step):
        t[r:r + step] = torch.randint(-128, 128, (min(step, rows - r), cols), dtype=torch.int8, device=gpu, generator=g)
    return t


def _rows_around(rows, per_row, *borders):
    """The first and last rows and those on both sides of the given offsets."""
    pick = {0, 1, rows // 2, rows - 2, rows - 1}
    for b in borders:
        for d in (-1, 0, 1):
            if 0 <= b // per_row + d < rows:
                pick.add(b // per_row + d)
    return sorted(pick)


def _ints(t):
    return t.cpu().numpy().astype(np.int64)


@pytest.mark.parametrize("few", [24, 300])
@pytest.mark.parametrize("tall", ["a", "b"])
def test_product_operand_past_4_gib(gpu, tall, few):
    """a or b of 5.2 GB. Sums of int8 products are exact in int32; with scales 1 the fp32 output is the sum rounded once."""
    import torch
    n, K = 40009, 131056
    assert n * K > 2 ** 32
    _say(f"[large product] {tall} {n} x {K}, other {few}")
    x, y = _codes(gpu, n, K, 1), _codes(gpu, few, K, 2)
    sx, sy = torch.ones(n, device=gpu), torch.ones(few, device=gpu)
    out = moe.gemm_i8(x, sx, y, sy, out_dtype=torch.float32) if tall == "a" else \
        moe.gemm_i8(y, sy, x, sx, out_dtype=torch.float32).t()
    torch.cuda.synchronize()
    yi = _ints(y).astype(np.float64)
    pick = _rows_around(n, K, 2 ** 31, 2 ** 32)
    want = _ints(x[pick]).astype(np.float64) @ yi.T                   # below 2^31: exact in fp64
    assert np.array_equal(out[pick].cpu().numpy(), want.astype(np.float32))


def test_gated_product_operand_past_4_gib(gpu):
    """w13 of 5.2 GB, whose up rows lie past 2^31 bytes: equal rows give equal outputs to a small call's."""
    import torch
    I, K, M = 20005, 131056, 40
    assert 2 * I * K > 2 ** 32
    _say(f"[large gated product] w13 {2 * I} x {K}")
    w, a = _codes(gpu, 2 * I, K, 3), _codes(gpu, M, K, 4)
    sa, sw = torch.ones(M, device=gpu), torch.full((2 * I,), 2.0 ** -20, device=gpu)
    h = moe.glu_i8(a, sa, w, sw)
    pick = _rows_around(I, K, 2 ** 31, 2 ** 32 - I * K)
    rows = torch.tensor(pick + [I + i for i in pick], device=gpu)
    want = moe.glu_i8(a, sa, w[rows], sw[:2 * len(pick)])
    torch.cuda.synchronize()
    assert torch.equal(h[:, pick], want)


@pytest.mark.parametrize("N", [16392, 16389])
def test_product_output_past_4_gib(gpu, N):
    """2^31 outputs, 4.3 GB (aligned rows and not), added in place."""
    import torch
    M, K = 131101, 16
    assert M * N > 2 ** 31
    _say(f"[large output] {M} x {N}")
    a, b = _codes(gpu, M, K, 5), _codes(gpu, N, K, 6)
    sa, sb = torch.full((M,), 2.0 ** -10, device=gpu), torch.ones(N, device=gpu)
    out = torch.full((M, N), 2.0, dtype=torch.bfloat16, device=gpu)
    moe.gemm_i8(a, sa, b, sb, add=out, out=out)
    torch.cuda.synchronize()
    pick = _rows_around(M, N, 2 ** 30, 2 ** 31)
    want = torch.from_numpy(_ints(a[pick]) @ _ints(b).T).double() * 2.0 ** -10 + 2       # 19 bits: exact in fp32
    assert torch.equal(out[pick].cpu(), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("T,H", [(262149, 16384), (524420, 8191), (2100000, 2048)])
def test_rows_past_2_to_the_32(gpu, T, H):
    """Norm, quantizer and the way back over 4.3e9 values, on rows of each kind: workgroup, shifted, wave."""
    import torch
    assert T * H > 2 ** 32
    _say(f"[large rows] {T} x {H}")
    x = torch.empty(T, H, dtype=torch.bfloat16, device=gpu)
    for r in range(0, T, 16384):
        x[r:r + 16384].normal_(generator=None)
    w = 1 + 0.1 * torch.randn(H, device=gpu)
    pick = _rows_around(T, H, 2 ** 31, 2 ** 32)
    few = x[pick].contiguous()
    if H == 2048:                                                     # (the wave form is taken from 1024 rows on)
        few = few.repeat(1024, 1)
    y, total, codes, scales = moe.norm(x, w, 1e-6, res=x, q_mode=moe.Q_I8_ROW)
    y1, t1, c1, s1 = moe.norm(few, w, 1e-6, res=few, q_mode=moe.Q_I8_ROW)
    n = len(pick)
    torch.cuda.synchronize()
    for big, small in ((y, y1), (total, t1), (codes, c1), (scales, s1)):
        assert torch.equal(big[pick], small[:n])
    if H % 128 == 0:
        del y, codes
        y, _, codes, scales = moe.norm(x, None, 1e-6, q_mode=moe.Q_FP8_G128_POW2)
        y1, _, c1, s1 = moe.norm(few, None, 1e-6, q_mode=moe.Q_FP8_G128_POW2)
        for big, small in ((y, y1), (codes, c1), (scales, s1)):
            assert torch.equal(big[pick], small[:n])
        back = moe.dequant_rows(codes, scales, out=total)
        assert torch.equal(back[pick], moe.dequant_rows(c1, s1)[:n])
    codes, scales = moe.quant_rows(x)
    c1, s1 = moe.quant_rows(few)
    assert torch.equal(codes[pick], c1[:n]) and torch.equal(scales[pick], s1[:n])
    if H % 8 == 0:
        back = moe.dequant_rows(codes, scales, out=total)
        assert torch.equal(back[pick], moe.dequant_rows(c1, s1)[:n])
    else:
        with pytest.raises(moe.MoeError):                             # one thread a value: below 2^31
            moe.dequant_rows(codes, scales)


@pytest.mark.parametrize("M,N", [((1 << 26) + 1, 1), ((1 << 25) + 3, 5), (1, (1 << 26) + 3), (2, (1 << 25) + 1)])
def test_products_one_side_of_which_is_very_long(gpu, M, N):
    """Outputs narrower than a lane's columns, and a million tiles in a row."""
    import torch
    K = 16
    _say(f"[long product] {M} x {N}")
    a, b = _codes(gpu, M, K, 7), _codes(gpu, N, K, 8)
    sa, sb = torch.ones(M, device=gpu), torch.ones(N, device=gpu)
    add = torch.full((M, N), 0.5, device=gpu)
    out = moe.gemm_i8(a, sa, b, sb, add=add, out_dtype=torch.float32)
    want = add.clone()                                                # below 2^19 and a half: exact in fp32
    for k in range(K):
        want += a[:, k:k + 1].float() * b[:, k].float()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    w13 = torch.cat([b, b.flip(0)])
    h = moe.glu_i8(a, sa * 2.0 ** -9, w13, torch.cat([sb, sb]))
    pick = _rows_around(M, 1, 1 << 25) if M > N else sorted({0, M - 1})
    few = moe.glu_i8(a[pick].contiguous(), sa[:len(pick)] * 2.0 ** -9, w13, torch.cat([sb, sb]))
    torch.cuda.synchronize()
    assert torch.equal(h[pick], few)


@pytest.mark.parametrize("M,N", [(1 << 30, 1), (1, 1 << 30), ((1 << 29) + 77, 3)])
def test_products_of_the_longest_sides(gpu, M, N):
    """2^30 rows of either operand: more small tiles than a launch has threads for."""
    import torch
    K = 16
    _say(f"[longest product] {M} x {N}")
    a, b = _codes(gpu, M, K, 9), _codes(gpu, N, K, 10)
    sa, sb = torch.full((M,), 2.0 ** -4, device=gpu), torch.ones(N, device=gpu)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=gpu)
    moe.gemm_i8(a, sa, b, sb, out=out)
    tall, few, got = (a, b, out) if M > N else (b, a, out.t())
    for r in range(0, max(M, N), 1 << 26):
        part = tall[r:r + (1 << 26)].float()
        for j in range(few.shape[0]):
            want = torch.zeros(part.shape[0], device=gpu)             # below 2^19: exact in fp32
            for k in range(K):
                want += part[:, k] * few[j, k].float()
            assert torch.equal(got[r:r + (1 << 26), j], (want * 2.0 ** -4).to(torch.bfloat16)), (r, j)


def test_gated_product_of_the_longest_side(gpu):
    """2^29 gate and as many up rows: equal rows give equal outputs to a small call's."""
    import torch
    I, K, M = 1 << 29, 16, 2
    _say(f"[longest gated product] {M} x {I}")
    w, a = _codes(gpu, 2 * I, K, 11), _codes(gpu, M, K, 12)
    sa, sw = torch.ones(M, device=gpu), torch.full((2 * I,), 2.0 ** -9, device=gpu)
    h = torch.full((M, I), 7.0, dtype=torch.bfloat16, device=gpu)
    moe.glu_i8(a, sa, w, sw, out=h)
    for r in sorted({0, 1 << 20, I // 2 - 50, I - (1 << 16)}):
        n = min(1 << 16, I - r)
        few = torch.cat([w[r:r + n], w[I + r:I + r + n]])
        assert torch.equal(h[:, r:r + n], moe.glu_i8(a, sa, few, sw[:2 * n])), r
