"""The FP8 products with a scale per block of 128 (moe_gemm_fp8, moe_glu_fp8)
against the fp64 oracle.

Tolerances, with u = 2^-24, mag the sum of the terms' magnitudes:
* a block's sum: 127 additions inside a matrix instruction that may drop bits
  instead of rounding, 2 u each: 254 u mag; one multiply-add per block, at most
  K / 128 of them and 8 joins of partial sums, u each; bias and addend u each:
  (254 + K / 128 + 10) u mag. The output type adds its half step, bf16 2^-8.
* bf16 outputs come from the FP8 instruction, whose 128 products are aligned
  at the largest one's exponent e and lose what lies below 2^(e - 13): less than
  2^-13 of the largest product each, 128 2^-13 = 2^-6 of it in a block's sum.
  "largest" adds that over the blocks.
* small whole codes under powers of two have exact sums in any order: fp32
  outputs are equal, bf16 outputs the exact value rounded.
* glu: with g and u off by dg and du: silu' lies in [-0.1, 1.1], so h is off by
  1.1 dg |u| + |silu(g)| du, plus (4 |g| + 16) u |h| for the exponential, the
  reciprocal and the products (as for the int8 product), plus the second-order
  1.1 dg du and the output's half step.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import dense

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HB = 2.0 ** -8


def _say(*a):
    print(*a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


def _dev(a, dev, shift=0):
    """An array on the device, `shift` elements past a 16-byte boundary."""
    import torch
    a = torch.from_numpy(np.ascontiguousarray(a))
    buf = torch.empty(a.numel() + shift, dtype=a.dtype, device=dev)
    t = buf[shift:].view(a.shape)
    t.copy_(a)
    return t


def _blocks(n):
    return (n + 127) // 128


def _codes(r, rows, K):
    """Random finite e4m3 codes of both signs, subnormals among them."""
    c = r.integers(0, 0x7F, size=(rows, K)).astype(np.uint8)
    return c | (r.integers(0, 2, size=(rows, K)).astype(np.uint8) << 7)


# e4m3 codes of -3 .. 3
WHOLE = np.array([0xC4, 0xC0, 0xB8, 0x00, 0x38, 0x40, 0x44], dtype=np.uint8)


def _operands(r, M, N, K, nb, exact):
    if exact:
        a, b = WHOLE[r.integers(0, 7, size=(M, K))], WHOLE[r.integers(0, 7, size=(N, K))]
        sa = r.integers(126, 129, size=(M, _blocks(K))).astype(np.uint8)
        sb = np.exp2(r.integers(-2, 2, size=(nb, _blocks(K)))).astype(np.float32)
    else:
        a, b = _codes(r, M, K), _codes(r, N, K)
        sa = r.integers(117, 123, size=(M, _blocks(K))).astype(np.uint8)
        sb = (0.02 / K ** 0.5 * np.exp(0.5 * r.normal(size=(nb, _blocks(K))))).astype(np.float32)
    return a, sa, b, sb


def _within(name, got, ref, tol):
    d = np.abs(got - ref)
    worst = float(np.max(d / np.maximum(tol, 1e-300)))
    _say(f"    {name}: worst |got - exact| / tolerance {worst:.3f}")
    assert np.all(d <= tol), f"{name}: {int((d > tol).sum())} of {d.size} outside"


SHAPES = [(1, 1, 16), (1, 2048, 2048), (1, 17, 8192), (2, 300, 144), (7, 64, 128), (16, 129, 112), (32, 2048, 512), (31, 33, 1040),
          (33, 128, 4112), (64, 513, 256), (65, 127, 400), (100, 1000, 2064), (128, 128, 128), (130, 260, 640), (255, 257, 272),
          (256, 256, 256), (257, 511, 2048), (333, 1000, 4112), (700, 2048, 384), (1030, 770, 528), (2049, 1300, 1152),
          (4100, 2048, 256), (5000, 2056, 16), (1500, 1100, 6160), (4100, 2100, 4112), (4096, 2048, 4608), (1024, 2048, 2304)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("f32", [True, False])
def test_gemm_exact_sums(gpu, M, N, K, f32):
    import torch
    r = np.random.default_rng([1, M, N, K])
    _say(f"[gemm_fp8 exact] {M} x {N} x {K} f32={f32}")
    a, sa, b, sb = _operands(r, M, N, K, _blocks(N), True)
    out = moe.gemm_fp8(*(_dev(x, gpu) for x in (a, sa, b, sb)), out_dtype=torch.float32 if f32 else None)
    torch.cuda.synchronize()
    _, ref = dense.gemm_fp8(a, sa, b, sb)
    if f32:
        assert np.array_equal(_f64(out), ref)
    else:
        assert torch.equal(out.cpu(), torch.from_numpy(ref).to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bias,add,f32,shift", [(True, True, True, 0), (False, True, False, 0), (True, True, False, 3)])
def test_gemm(gpu, M, N, K, bias, add, f32, shift):
    import torch
    r = np.random.default_rng([2, M, N, K, bias, f32])
    _say(f"[gemm_fp8] {M} x {N} x {K} bias={bias} add={add} f32={f32} shift={shift}")
    a, sa, b, sb = _operands(r, M, N, K, _blocks(N), False)
    bs = r.normal(size=N).astype(np.float32) if bias else None
    ot = torch.float32 if f32 else torch.bfloat16
    plus = torch.from_numpy(r.normal(size=(M, N)).astype(np.float32)).to(ot) if add else None
    buf = torch.empty(M * N + shift, dtype=ot, device=gpu)
    out = buf[shift:].view(M, N)
    ag = None
    if add:
        ag = torch.empty(M * N + shift, dtype=ot, device=gpu)[shift:].view(M, N)
        ag.copy_(plus)
    ops = (_dev(a, gpu), _dev(sa, gpu, shift), _dev(b, gpu), _dev(sb, gpu, shift))
    got = moe.gemm_fp8(*ops, bias=None if bs is None else _dev(bs, gpu, shift), add=ag, out=out)
    torch.cuda.synchronize()
    assert got is out
    mag, ref = dense.gemm_fp8(a, sa, b, sb, bs, None if plus is None else plus.double().numpy())
    tol = (254 + K / 128 + 10) * U * mag + (0 if f32 else 2.0 ** -6 * dense.fp8_largest(a, sa, b, sb))
    _within("out", _f64(out), ref, tol + (0 if f32 else HB * (np.abs(ref) + tol)))
    again = moe.gemm_fp8(*ops, bias=None if bs is None else _dev(bs, gpu), add=ag, out_dtype=ot)
    if add:                                                       # the addend's own memory
        moe.gemm_fp8(*ops, bias=None if bs is None else _dev(bs, gpu), add=ag, out=ag)
        torch.cuda.synchronize()
        assert torch.equal(ag, got)
    assert torch.equal(again, got)


@pytest.mark.parametrize("M,I,K", [(1, 1, 16), (1, 512, 2048), (8, 512, 2048), (5, 100, 272), (33, 129, 128), (64, 768, 2048), (129, 200, 400),
                                   (300, 512, 1040), (520, 130, 2048), (1025, 512, 256), (3000, 700, 144), (4099, 512, 384), (2500, 700, 2320),
                                   (4096, 1024, 2176)])
def test_glu(gpu, M, I, K):
    import torch
    r = np.random.default_rng([3, M, I, K])
    _say(f"[glu_fp8] {M} x {I} x {K}")
    for exact in (True, False):
        a, sa, w, s = _operands(r, M, 2 * I, K, 2 * _blocks(I), exact)
        if exact:
            s *= np.float32(2.0 ** -6)
        h = moe.glu_fp8(*(_dev(x, gpu) for x in (a, sa, w, s)))
        torch.cuda.synchronize()
        g, u, mg, mu, ref = dense.glu_fp8(a, sa, w, s)
        e, d = (0, 0) if exact else ((254 + K / 128 + 8) * U, 2.0 ** -6)
        half = _blocks(I)
        dg, du = e * mg + d * dense.fp8_largest(a, sa, w[:I], s[:half]), e * mu + d * dense.fp8_largest(a, sa, w[I:], s[half:])
        tol = 1.1 * dg * np.abs(u) + (np.abs(g) / (1 + np.exp(-np.clip(g, -700, 700))) + 1.1 * dg) * du + (4 * np.abs(g) + 16) * U * np.abs(ref)
        _within(f"h (exact {exact})", _f64(h), ref, tol + HB * (np.abs(ref) + tol) + 2.0 ** -120)


@pytest.mark.parametrize("M,N,K", [(3, 200, 144), (40, 130, 80), (200, 300, 400), (600, 520, 272), (3000, 2050, 144)])
def test_nothing_of_other_rows_enters(gpu, M, N, K):
    """NaN in a row of a or b, in its scales and behind the operands stays in that row's outputs, also where a
    load runs on into the next row (K no multiple of 128)."""
    import torch
    r = np.random.default_rng([4, M, N, K])
    a, sa, b, sb = _operands(r, M, N, K, _blocks(N), True)
    rows, cols = [1, M - 1], [0, N // 2]
    clean = dense.gemm_fp8(a, sa, b, sb)[1]
    a[rows[0]], a[rows[1], K - 1], b[cols[0]], b[cols[1], 0] = 0x7F, 0xFF, 0xFF, 0x7F

    def inside(x):
        big = torch.full((x.size + 4096,), 255 if x.dtype == np.uint8 else float("nan"), device=gpu,
                         dtype=torch.uint8 if x.dtype == np.uint8 else torch.float32)
        t = big[1024:1024 + x.size].view(x.shape)
        t.copy_(torch.from_numpy(x))
        return t
    out = moe.gemm_fp8(*(inside(x) for x in (a, sa, b, sb)), out_dtype=torch.float32)
    torch.cuda.synchronize()
    got = _f64(out)
    want = np.zeros((M, N), dtype=bool)
    want[rows], want[:, cols] = True, True
    assert np.array_equal(np.isnan(got), want)
    assert np.array_equal(got[~want], clean[~want])
    sa[M // 2, -1] = 255
    out = _f64(moe.gemm_fp8(*(inside(x) for x in (a, sa, b, sb)), out_dtype=torch.float32))
    want[M // 2] = True
    assert np.array_equal(np.isnan(out), want)
    sb[0, 0] = np.nan
    out = _f64(moe.gemm_fp8(*(inside(x) for x in (a, sa, b, sb)), out_dtype=torch.float32))
    want[:, :128] = True
    assert np.array_equal(np.isnan(out), want)


def test_glu_rows_of_gate_and_up_apart(gpu):
    """NaN in one gate row and one up row reaches their columns alone (I no multiple of 128)."""
    import torch
    r = np.random.default_rng(5)
    for M, I, K in ((5, 77, 144), (300, 200, 80), (2000, 321, 272)):
        a, sa, w, s = _operands(r, M, 2 * I, K, 2 * _blocks(I), True)
        s *= np.float32(2.0 ** -6)
        w[3], w[I + I - 1] = 0x7F, 0xFF
        h = _f64(moe.glu_fp8(*(_dev(x, gpu) for x in (a, sa, w, s))))
        torch.cuda.synchronize()
        want = np.zeros((M, I), dtype=bool)
        want[:, [3, I - 1]] = True
        assert np.array_equal(np.isnan(h), want)


def test_types_and_the_rows_that_the_library_writes(gpu):
    """float8 tensors are taken like their bytes, and norm's and quant_act's rows as they come."""
    import torch
    r = np.random.default_rng(6)
    T, H, N = 37, 512, 200
    x = torch.from_numpy(r.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).to(gpu)
    _, _, b, sb = _operands(r, 1, N, H, _blocks(N), False)
    bd, sd = _dev(b, gpu), _dev(sb, gpu)
    for codes, scales in (moe.quant_act(x), moe.norm(x, None, 1e-6, q_mode=moe.Q_FP8_G128_POW2)[2:]):
        out = moe.gemm_fp8(codes, scales, bd, sd, out_dtype=torch.float32)
        same = moe.gemm_fp8(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), bd.view(torch.float8_e4m3fn), sd,
                            out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(out, same)
        mag, ref = dense.gemm_fp8(codes.cpu().numpy(), scales.cpu().numpy(), b, sb)
        _within("out", _f64(out), ref, (254 + H / 128 + 10) * U * mag)


def test_extreme_scales(gpu):
    """Powers of two from the smallest to the largest whose sums stay in fp32's range are exact."""
    import torch
    r = np.random.default_rng(7)
    for M, N, K in ((4, 40, 256), (300, 300, 256)):
        a, sa, b, sb = _operands(r, M, N, K, _blocks(N), True)
        sa[:, 0], sa[:, 1] = 20, 230
        sb[:, 0], sb[:, 1] = 2.0 ** 100, 2.0 ** -110
        out = moe.gemm_fp8(*(_dev(x, gpu) for x in (a, sa, b, sb)), out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert np.array_equal(_f64(out), dense.gemm_fp8(a, sa, b, sb)[1])


def test_shared_expert(gpu):
    """The three calls' result, and a token's row of a norm through the expert and into the next residual."""
    import torch
    r = np.random.default_rng(8)
    for T, H, I in ((1, 256, 128), (33, 512, 256), (400, 1024, 512)):
        x = torch.from_numpy(r.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).to(gpu)
        _, _, w13, s13 = _operands(r, 1, 2 * I, H, 2 * _blocks(I), False)
        _, _, w2, s2 = _operands(r, 1, H, I, _blocks(H), False)
        w13, s13, w2, s2 = (_dev(v, gpu) for v in (w13, s13, w2, s2))
        routed = torch.from_numpy(r.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).to(gpu)
        _, _, a, sa = moe.norm(x, None, 1e-6, q_mode=moe.Q_FP8_G128_POW2, with_y=False)
        h = moe.glu_fp8(a, sa, w13, s13)
        hq, hs = moe.quant_act(h)
        want = moe.gemm_fp8(hq, hs, w2, s2, add=routed)
        got = moe.shared_expert_fp8(a, sa, w13, s13, w2, s2, add=routed)
        side = torch.cuda.Stream(gpu)
        side.wait_stream(torch.cuda.current_stream(gpu))
        there = moe.shared_expert_fp8(a, sa, w13, s13, w2, s2, add=routed, stream=side)
        inplace = routed.clone()
        assert moe.shared_expert_fp8(a, sa, w13, s13, w2, s2, add=inplace, out=inplace) is inplace
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(there, want) and torch.equal(inplace, want)
        mag, ref = dense.gemm_fp8(hq.cpu().numpy(), hs.cpu().numpy(), w2.cpu().numpy(), s2.cpu().numpy(), None, _f64(routed))
        tol = (254 + I / 128 + 10) * U * mag + 2.0 ** -6 * dense.fp8_largest(*(v.cpu().numpy() for v in (hq, hs, w2, s2)))
        _within("out", _f64(got), ref, tol + HB * (np.abs(ref) + tol))


def test_captured_and_replayed(gpu):
    import torch
    r = np.random.default_rng(9)
    runs = []
    for M, N, K in ((1, 2048, 512), (33, 300, 272), (500, 512, 1024), (4096, 512, 512)):
        a, sa, b, sb = (_dev(v, gpu) for v in _operands(r, M, N, K, _blocks(N), False))
        runs.append((a, sa, b, sb, torch.empty(M, N, dtype=torch.bfloat16, device=gpu), torch.empty(M, N // 2, dtype=torch.bfloat16, device=gpu),
                     _dev(r.random((2 * _blocks(N // 2), _blocks(K))).astype(np.float32) * 0.001, gpu)))
    want = [(moe.gemm_fp8(a, sa, b, sb), moe.glu_fp8(a, sa, b, s13)) for a, sa, b, sb, _, _, s13 in runs]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for a, sa, b, sb, out, h, s13 in runs:
            moe.gemm_fp8(a, sa, b, sb, out=out)
            moe.glu_fp8(a, sa, b, s13, out=h)
    for k in range(4):
        for *_, out, h, _ in runs:
            out.zero_()
            h.zero_()
        g.replay()
        torch.cuda.synchronize()
        for (w, wh), (*_, out, h, _) in zip(want, runs):
            assert torch.equal(w, out) and torch.equal(wh, h), k


def test_refusals(gpu):
    import torch
    u8 = dict(dtype=torch.uint8, device=gpu)
    f32 = dict(dtype=torch.float32, device=gpu)
    a, sa, b, sb = torch.zeros(4, 256, **u8), torch.zeros(4, 2, **u8), torch.zeros(300, 256, **u8), torch.zeros(3, 2, **f32)
    moe.gemm_fp8(a, sa, b, sb)
    s13 = torch.zeros(4, 2, **f32)
    moe.glu_fp8(a, sa, b, s13)
    for bad in ((a.cpu(), sa, b, sb), (a.to(torch.int8), sa, b, sb), (a.t(), sa, b, sb), (a[:, ::2], sa, b, sb), (a[0], sa, b, sb),
                (a[:0], sa[:0], b, sb), (a, sa[:, :1], b, sb), (a, sa[:, :1].contiguous(), b, sb), (a, sa.float(), b, sb), (a, None, b, sb),
                (a, sa, b[:, :128].contiguous(), sb), (a, sa, b, sb[:2]), (a, sa, b, sb.t()), (a, sa, b, sb.double()), (a, sa, None, sb),
                (a[:, :24].contiguous(), sa[:, :1].contiguous(), b[:, :24].contiguous(), sb[:, :1].contiguous())):
        with pytest.raises(moe.MoeError):
            moe.gemm_fp8(*bad)
    for kw in ({"bias": torch.zeros(4, **f32)}, {"add": torch.zeros(4, 300, **f32)}, {"out": torch.zeros(300, 4, **f32)},
               {"out_dtype": torch.float16}, {"out": torch.zeros(4, 300, **f32), "out_dtype": torch.bfloat16}):
        with pytest.raises(moe.MoeError):
            moe.gemm_fp8(a, sa, b, sb, **kw)
    for bad in ((a, sa, b[:299], s13), (a, sa, b, sb), (a, sa, b, torch.zeros(3, 2, **f32)), (a, sa, b[:, :128].contiguous(), s13)):
        with pytest.raises(moe.MoeError):
            moe.glu_fp8(*bad)
    big = torch.zeros(4 * 256 + 8, **u8)
    with pytest.raises(moe.MoeError):
        moe.gemm_fp8(big[8:].view(4, 256), sa, b, sb)
    with pytest.raises(moe.MoeError):                             # rows back to e4m3 need whole groups
        moe.shared_expert_fp8(a, sa, torch.zeros(200, 256, **u8), torch.zeros(2, 2, **f32), torch.zeros(256, 100, **u8), torch.zeros(2, 1, **f32))
