"""bf16 outputs and the gated form of the FP8 products, whose scale bytes are an
operand of the matrix instruction: NaN bytes, the smallest and the largest
powers of two, and the loss of their sums.

* Small whole codes under powers of two have exact sums: outputs are the exact
  value, rounded once (the gated form: tolerance of test_gpu_fp8.py with exact g, u).
* The loss: out1 + out2, with out2 the product that has -out1 as its addend, is
  the product's sum before rounding, off by out2's own rounding: sum - out1 is at
  most 2^-8 of the sum and exact in fp32, its rounding 2^-8 of that. With the loss
  L of the norm that the header states (less than 1e-4, heavy tails or not) and the fp32 sums'
  (254 + K / 128 + 10) 2^-24 |magnitudes|, the difference's norm is at most
  (L + 2^-16) of the reference's, plus that of the fp32 sums. out1 itself is the
  nearest bf16 of its sum, and no farther from it than the rounded reference is,
  which is off by the rounded reference's error and the loss: out1's error is at
  most the rounded reference's and twice the loss.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import dense
from test_gpu_fp8 import HB, U, _blocks, _dev, _f64, _operands, _say, _within

LOSS = 1e-4                                                       # of the outputs' norm

# a launch of every tile: 32x32, 32x64, 64x64, 128x128 (few, many), 256x256; whole lines and odd widths
SHAPES = [(3, 200, 144), (40, 130, 80), (200, 300, 400), (300, 1000, 2048), (500, 2048, 272), (1024, 2048, 512), (1500, 1100, 656),
          (4096, 2048, 512), (4100, 2050, 528), (8200, 2048, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_nan_scale_bytes(gpu, M, N, K):
    """A row's byte of 255 makes the row NaN, also beside codes of zero (as norm writes bad rows); a block's NaN its columns."""
    import torch
    _say(f"[scales, NaN] {M} x {N} x {K}")
    r = np.random.default_rng([31, M, N, K])
    a, sa, b, sb = _operands(r, M, N, K, _blocks(N), True)
    kb = _blocks(K)
    bad = {0: (0, False), M // 2: (kb - 1, True), M - 1: (kb // 2, True)}
    for row, (j, zero) in bad.items():
        sa[row, j] = 255
        if zero:
            a[row, 128 * j:128 * (j + 1)] = 0
    out = _f64(moe.gemm_fp8(*(_dev(x, gpu) for x in (a, sa, b, sb))))
    ref = dense.gemm_fp8(a, sa, b, sb)[1]
    want = np.zeros((M, N), dtype=bool)
    want[list(bad)] = True
    assert np.array_equal(np.isnan(out), want)
    rounded = torch.from_numpy(np.where(want, 0, ref)).to(torch.bfloat16).double().numpy()
    assert np.array_equal(np.where(want, 0, out), rounded)
    sb[-1, 0] = np.nan
    want[:, 128 * (_blocks(N) - 1):] = True
    assert np.array_equal(np.isnan(_f64(moe.gemm_fp8(*(_dev(x, gpu) for x in (a, sa, b, sb))))), want)

    inter = N // 2
    a, sa, w, s = _operands(r, M, 2 * inter, K, 2 * _blocks(inter), True)
    s *= np.float32(2.0 ** -6)
    for row, (j, zero) in bad.items():
        sa[row, j] = 255
        if zero:
            a[row, 128 * j:128 * (j + 1)] = 0
    want = np.zeros((M, inter), dtype=bool)
    want[list(bad)] = True
    assert np.array_equal(np.isnan(_f64(moe.glu_fp8(*(_dev(x, gpu) for x in (a, sa, w, s))))), want)
    s[-1, kb - 1] = np.nan                                        # the last block of the up rows
    want[:, 128 * (_blocks(inter) - 1):] = True
    assert np.array_equal(np.isnan(_f64(moe.glu_fp8(*(_dev(x, gpu) for x in (a, sa, w, s))))), want)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_rows_of_a_norm(gpu, bad):
    """norm's codes of zero with a NaN byte make the product's row NaN, and that row alone."""
    import torch
    r = np.random.default_rng(32)
    for M, N, H in ((3, 256, 512), (700, 1024, 256), (4096, 2048, 512)):
        x = torch.from_numpy(r.normal(size=(M, H)).astype(np.float32)).to(torch.bfloat16)
        x[M // 2, H - 3] = bad
        _, _, codes, scales = moe.norm(x.to(gpu), None, 1e-6, q_mode=moe.Q_FP8_G128_POW2, with_y=False)
        _, _, b, sb = _operands(r, 1, N, H, _blocks(N), False)
        bd, sd = _dev(b, gpu), _dev(sb, gpu)
        want = np.zeros(M, dtype=bool)
        want[M // 2] = True
        for out in (moe.gemm_fp8(codes, scales, bd, sd), moe.glu_fp8(codes, scales, bd, sd)):
            nan = np.isnan(_f64(out))
            assert np.array_equal(nan.all(axis=1), want) and np.array_equal(nan.any(axis=1), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("first,last,s0,s1", [(20, 230, 100, -110), (1, 254, 120, -126), (3, 250, 126, -120)])
def test_extreme_scales(gpu, M, N, K, first, last, s0, s1):
    """Powers of two from the smallest to the largest whose block sums are normal values of fp32: a row has one code of +-1 in
    each block, which meets weights of -1, 0 and 1."""
    import torch
    _say(f"[scales, extreme] {M} x {N} x {K} {first}, {last}")
    r = np.random.default_rng([33, M, N, K, first])
    kb = _blocks(K)

    def one_of_a_block(rows):
        c = np.zeros((rows, K), dtype=np.uint8)
        for j in range(kb):
            at = 128 * j + r.integers(0, min(16, K - 128 * j), size=rows)
            c[np.arange(rows), at] = np.where(r.random(rows) < 0.5, 0x38, 0xB8)          # +-1
        return c
    a, b = one_of_a_block(M), WEIGHTS[r.integers(0, 3, size=(N, K))]
    sa = r.integers(126, 129, size=(M, kb)).astype(np.uint8)
    sb = np.exp2(r.integers(-2, 2, size=(_blocks(N), kb))).astype(np.float32)
    sa[:, 0], sb[:, 0] = first, 2.0 ** s0
    if kb > 1:
        sa[:, -1], sb[:, -1] = last, 2.0 ** s1
    out = moe.gemm_fp8(*(_dev(x, gpu) for x in (a, sa, b, sb)))
    torch.cuda.synchronize()
    ref = dense.gemm_fp8(a, sa, b, sb)[1]
    assert torch.equal(out.cpu(), torch.from_numpy(ref).to(torch.bfloat16))


WEIGHTS = np.array([0xB8, 0x00, 0x38], dtype=np.uint8)            # -1, 0, 1


@pytest.mark.gpu
@pytest.mark.parametrize("M,I,K", [(3, 100, 256), (130, 300, 272), (4096, 1024, 256)])
def test_extreme_scales_gated(gpu, M, I, K):
    import torch
    r = np.random.default_rng([34, M])
    a, sa, w, s = _operands(r, M, 2 * I, K, 2 * _blocks(I), True)
    sa[:, 0], sa[:, 1] = 20, 230
    s[:, 0], s[:, 1] = 2.0 ** 101, 2.0 ** -109
    h = moe.glu_fp8(*(_dev(x, gpu) for x in (a, sa, w, s)))
    torch.cuda.synchronize()
    g, u, _, _, ref = dense.glu_fp8(a, sa, w, s)
    # sums of the third block take g to -227: below -87.3 the sigmoid lies below fp32's smallest normal value 2^-126, where the
    # hardware's reciprocal gives 0, and below -88.8 its exponential is infinite, with the same 0: h is off by the sigmoid
    # that is lost times |g u|, less than 2^-126 |g u|
    tol = (4 * np.abs(g) + 16) * U * np.abs(ref) + 2.0 ** -126 * np.abs(g * u)
    _within("h", _f64(h), ref, tol + HB * (np.abs(ref) + tol) + 2.0 ** -120)


@pytest.mark.gpu
def test_past_the_largest_fp32(gpu):
    """A block's sum past fp32's largest is infinite, with its sign, in bf16 and fp32 outputs."""
    import torch
    for M, N, K in ((2, 64, 128), (300, 512, 256), (4096, 2048, 256)):
        a = torch.full((M, K), 0x7E, dtype=torch.uint8, device=gpu)                      # 448
        b = torch.full((N, K), 0x7E, dtype=torch.uint8, device=gpu)
        b[N // 2:] = 0xFE
        sa = torch.full((M, _blocks(K)), 127, dtype=torch.uint8, device=gpu)
        sa[0] = 254
        sb = torch.full((_blocks(N), _blocks(K)), 2.0 ** -100, device=gpu)
        for dt in (torch.bfloat16, torch.float32):
            out = moe.gemm_fp8(a, sa, b, sb, out_dtype=dt)
            inf = torch.full((N,), float("inf"), device=gpu, dtype=dt)
            inf[N // 2:] = -float("inf")
            assert torch.equal(out[0], inf) and bool(torch.isfinite(out[1:]).all()), (M, dt)


# ---------------------------------------------------------------- the sums' loss
def _values(r, rows, K, tails):
    """Codes of normal values whose group's largest of 128 is near 2.6 deviations, as quantized rows are; with tails: of
    normal values times e^(1.5 n), n normal too, the group's largest at 448."""
    import torch
    x = r.normal(size=(rows, K))
    if tails:
        x *= np.exp(1.5 * r.normal(size=(rows, K)))
        top = np.maximum.reduceat(np.abs(x), np.arange(0, K, 128), axis=1)
        x *= np.repeat(448 / top, 128, axis=1)[:, :K]
    else:
        x *= 110
    return torch.from_numpy(np.clip(x, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _value_operands(r, M, N, K, nb, tails=False):
    sa = r.integers(118, 122, size=(M, _blocks(K))).astype(np.uint8)
    sb = (0.002 * (0.5 + r.random(size=(nb, _blocks(K))))).astype(np.float32)
    return _values(r, M, K, tails), sa, _values(r, N, K, tails), sb


def _norm(x):
    return float(np.sqrt(np.sum(np.square(x))))


def _bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def _close(name, got, ref, loss, rounded):
    """The norm of got's error against `loss` (a norm): alone, or as the bf16 nearest to a sum with that loss."""
    limit = _norm(_bf16(ref) - ref) + 2 * loss if rounded else loss
    d = _norm(got - ref)
    _say(f"    {name}: error {d / _norm(ref):.2e} of the norm, limit {limit / _norm(ref):.2e}")
    assert d <= limit, f"{name}: {d / _norm(ref):.3e} of the norm, limit {limit / _norm(ref):.3e}"


LOSS_SHAPES = [(1, 2048, 2048), (32, 512, 2048), (128, 300, 4112), (300, 512, 8192), (1024, 2048, 1024), (2100, 2048, 1152)]


def _limits(K, mag, ref):
    return LOSS * _norm(ref) + (254 + K / 128 + 10) * U * _norm(mag)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", LOSS_SHAPES)
@pytest.mark.parametrize("tails", [False, True])
def test_loss_of_bf16_sums(gpu, M, N, K, tails):
    _say(f"[loss] {M} x {N} x {K} tails={tails}")
    r = np.random.default_rng([35, M, N, K])
    a, sa, b, sb = _value_operands(r, M, N, K, _blocks(N), tails)
    ops = [_dev(x, gpu) for x in (a, sa, b, sb)]
    one = moe.gemm_fp8(*ops)
    two = moe.gemm_fp8(*ops, add=-one)
    mag, ref = dense.gemm_fp8(a, sa, b, sb)
    loss = _limits(K, mag, ref)
    _close("sum", _f64(one) + _f64(two), ref, loss + 2.0 ** -16 * _norm(ref), False)
    _close("out", _f64(one), ref, loss, True)


@pytest.mark.gpu
@pytest.mark.parametrize("M,I,K", [(8, 512, 2048), (300, 300, 1040), (2100, 512, 2048)])
def test_loss_of_the_gated_form(gpu, M, I, K):
    """h is off by 1.1 |u| dg + |silu(g)| du + the second order, with dg and du of the loss's norm spread over the outputs (a
    factor of 4 for how unevenly: they follow g's and u's blocks, not one another), and (4 |g| + 16) u |h|."""
    _say(f"[loss, gated] {M} x {I} x {K}")
    r = np.random.default_rng([36, M, I, K])
    a, sa, w, s = _value_operands(r, M, 2 * I, K, 2 * _blocks(I))
    s *= np.float32(0.1)
    h = moe.glu_fp8(*(_dev(x, gpu) for x in (a, sa, w, s)))
    g, u, mg, mu, ref = dense.glu_fp8(a, sa, w, s)
    dg, du = _limits(K, mg, g) / g.size ** 0.5, _limits(K, mu, u) / u.size ** 0.5
    _close("h", _f64(h), ref, 4 * (1.1 * dg * _norm(u) + du * _norm(g / (1 + np.exp(-g))) + 1.1 * dg * du * g.size ** 0.5)
           + _norm((4 * np.abs(g) + 16) * U * ref), True)


@pytest.mark.parametrize("noise", [0.01, 0.003])
def test_the_limits_find_noise(noise):
    """The reference with normal noise of that share of its deviation, rounded, is outside both limits (no GPU)."""
    for M, N, K in ((32, 512, 2048), (128, 300, 4112)):
        r = np.random.default_rng([37, M])
        mag, ref = dense.gemm_fp8(*_value_operands(r, M, N, K, _blocks(N)))
        loss = _limits(K, mag, ref)
        _close("out", _bf16(ref * (1 + LOSS * np.sign(r.normal(size=ref.shape)))), ref, loss, True)
        sum_ = ref + noise * ref.std() * r.normal(size=ref.shape)
        one = _bf16(sum_)
        with pytest.raises(AssertionError):
            _close("out", one, ref, loss, True)
        with pytest.raises(AssertionError):
            _close("sum", one + _bf16(sum_ - one), ref, loss + 2.0 ** -16 * _norm(ref), False)
