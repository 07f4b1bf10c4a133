"""The dense 8-bit operators (moe_norm, moe_quant_rows, moe_gemm_i8,
moe_glu_i8) against the fp64 oracle, element by element.

Tolerances, with u = 2^-24 (half a step of fp32, relative to the value):
* norm: v is one rounding (u); a thread sums at most 64 squares in turn and
  the partial sums meet in 8 more additions, all terms positive, each square
  carrying 2 u from v: mean square within 75 u, so its inverse root within
  38 u + 2 u (the hardware's own) and, with two products and v's rounding,
  |y - exact| <= 44 u |y|: 64 u is used. An output type adds its half step:
  bf16 2^-8 |y|.
* int8 codes: t = y (127 / m) carries y's and m's errors and 2 roundings,
  |t - exact| <= 127 * 131 u < 1.0e-3, so |code - exact t| <= 0.501. Rows read
  from bf16 are exact, so quant_rows' t is within 2 roundings: 0.5 + 127 * 3 u.
* e4m3: half a step of the code, 2^-4 of its value, or 2^-10 where it is
  subnormal, plus 64 u of the value.
* gemm: the int32 sum is exact; three roundings (conversion, two products) and
  one per addition: 4 u (|p| + |bias| + |add|) with p the scaled product,
  plus bf16's half step of the output.
* glu: g and u carry 3 u each; e^-g by a base-2 exponential whose argument
  carries 4 u |g| absolutely (g's own error and one product), the rest of
  silu(g) u is at most 13 roundings: (4 |g| + 16) u relative, plus bf16's
  half step; below 2^-125 |g u| the exponential has overflowed.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import dense, e4m3_decode

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HB = 2.0 ** -8


def _say(*a):
    print(*a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


def _rng(*key):
    return np.random.default_rng(np.random.SeedSequence([77, *key]))


def _bf16(a, dev, shift=0):
    """fp array -> contiguous bf16 device tensor whose address is `shift` elements past a 16-byte boundary."""
    import torch
    a = np.ascontiguousarray(a, dtype=np.float32)
    buf = torch.empty(a.size + shift, dtype=torch.bfloat16, device=dev)
    t = buf[shift:].view(a.shape)
    t.copy_(torch.from_numpy(a).to(torch.bfloat16))
    return t


def _f32(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dev)


def _i8(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int8)).to(dev)


def _close(name, got, ref, tol):
    d = np.abs(got - ref)
    worst = float(np.max(d / tol)) if d.size else 0.0
    _say(f"    {name}: worst |got - exact| / tolerance {worst:.3f}")
    assert np.all(d <= tol), f"{name}: {int((d > tol).sum())} of {d.size} outside"


def _rows_values(r, T, H):
    x = r.normal(size=(T, H)) * np.exp(0.7 * r.normal(size=H))[None, :]
    if T > 2:
        x[1] = 0.0                                      # a row of zeros
        x[2] *= 2.0 ** -60                              # a very small row
    return x


def _check_codes_i8(codes, scales, y, slack, scale_tol):
    t, s = dense.i8_rows(y)
    c = codes.cpu().numpy().astype(np.float64)
    _close("scales", _f64(scales), s, np.abs(s) * scale_tol)
    _close("codes", c, t, np.full_like(t, 0.5 + slack))
    assert np.abs(c).max() <= 127


# ---------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 8), (4, 64), (33, 100), (2, 520), (7, 1111), (1023, 512), (1024, 512),
               (1025, 520), (1030, 1024), (1027, 2048), (6, 2056), (5, 4096), (3, 5000), (3, 8192), (2, 16383),
               (3, 16384)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("q", [0, 1, 2])
@pytest.mark.parametrize("res,w", [(True, True), (False, False)])
def test_norm(gpu, T, H, q, res, w):
    import torch
    if q == 2 and H % 128:
        pytest.skip("e4m3 groups need a multiple of 128 columns")
    r = _rng(T, H, q, res)
    _say(f"[norm] T={T} H={H} q={q} res={res} w={w}")
    x = _bf16(_rows_values(r, T, H), gpu)
    rs = _bf16(_rows_values(r, T, H), gpu) if res else None
    wt = _f32(1 + 0.2 * r.normal(size=H), gpu) if w else None
    y, total, codes, scales = moe.norm(x, wt, 1e-6, res=rs, q_mode=q)
    torch.cuda.synchronize()
    ry, rv = dense.rms_norm(_f64(x), None if wt is None else _f64(wt), 1e-6, None if rs is None else _f64(rs))
    tiny = 2.0 ** -133                                  # half a step of bf16's subnormals, and fp32's below it
    _close("y", _f64(y), ry, np.abs(ry) * (HB + 64 * U) + tiny)
    if res:
        _close("sum", _f64(total), rv, np.abs(rv) * (HB + 2 * U) + tiny)
    else:
        assert total is None
    if q == 0:
        assert codes is None and scales is None
    if q == 1:
        _check_codes_i8(codes, scales, ry, 1e-3, 66 * U)
    if q == 2:
        e = scales.cpu().numpy().astype(np.int64) - 127
        g = ry.reshape(T, H // 128, 128)
        m = np.abs(g).max(axis=2)
        # smallest s with m <= 448 2^s, decided wherever m is not within 64 u of the border
        with np.errstate(divide="ignore"):
            lo, hi = (np.where(m > 0, np.ceil(np.log2(np.where(m > 0, m, 1) * f / 448)), 0) for f in (1 - 65 * U, 1 + 65 * U))
        assert np.all((e >= lo) & (e <= hi))
        t = g / np.exp2(e)[:, :, None]
        c = e4m3_decode(codes.cpu().numpy()).reshape(t.shape)
        _close("e4m3", c, t, np.maximum(np.abs(t) * (2.0 ** -4 + 64 * U), 2.0 ** -10 + 64 * U))


@pytest.mark.parametrize("shift", [1, 4])
def test_norm_unaligned_rows(gpu, shift):
    import torch
    r = _rng(5, shift)
    x, rs = (_bf16(_rows_values(r, 9, 512), gpu, shift) for _ in range(2))
    y, total, codes, scales = moe.norm(x, None, 1e-5, res=rs, q_mode=moe.Q_I8_ROW)
    torch.cuda.synchronize()
    ry, rv = dense.rms_norm(_f64(x), None, 1e-5, _f64(rs))
    _close("y", _f64(y), ry, np.abs(ry) * (HB + 64 * U) + 2.0 ** -133)
    _check_codes_i8(codes, scales, ry, 1e-3, 66 * U)
    with pytest.raises(moe.MoeError):
        moe.norm(x, None, 1e-5, q_mode=moe.Q_FP8_G128_POW2)


@pytest.mark.parametrize("T,H", [(3, 512), (1100, 2048), (4, 4096), (3, 333)])
def test_norm_in_place_and_without_y(gpu, T, H):
    """sum in res's memory and y in x's give what separate outputs give, bit for bit."""
    import torch
    r = _rng(T, H, 6)
    x, rs = (_bf16(_rows_values(r, T, H), gpu) for _ in range(2))
    w = _f32(1 + 0.2 * r.normal(size=H), gpu)
    y0, s0, c0, f0 = moe.norm(x, w, 1e-6, res=rs, q_mode=moe.Q_I8_ROW)
    none, s1, c1, f1 = moe.norm(x, w, 1e-6, res=rs, q_mode=moe.Q_I8_ROW, with_y=False)
    assert none is None
    x2, r2 = x.clone(), rs.clone()
    y2, s2, c2, f2 = moe.norm(x2, w, 1e-6, res=r2, q_mode=moe.Q_I8_ROW, sum=r2, y=x2)
    torch.cuda.synchronize()
    assert y2 is x2 and s2 is r2
    for a, b in ((y0, y2), (s0, s1), (s0, s2), (c0, c1), (c0, c2), (f0, f1), (f0, f2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(4, 256), (1100, 256), (4, 201)])
def test_norm_nonfinite_rows(gpu, T, H):
    """A row (a group, for e4m3) that holds infinity or NaN has codes 0 and a NaN scale; the others are untouched."""
    import torch
    r = _rng(T, H, 8)
    x = _bf16(r.normal(size=(T, H)), gpu)
    good = moe.quant_rows(x)
    x[1, 3], x[2, H - 1], x[3, 0] = float("nan"), float("inf"), -float("inf")
    bad = moe.quant_rows(x)
    y, _, codes, scales = moe.norm(x, None, 1e-6, q_mode=moe.Q_I8_ROW)
    torch.cuda.synchronize()
    rest = [0] + list(range(4, T))
    for c, s in ((bad[0], bad[1]), (codes, scales)):
        assert torch.isnan(s[1:4]).all() and not c[1:4].any() and torch.isfinite(s[rest]).all()
    assert torch.equal(bad[0][rest], good[0][rest]) and torch.equal(bad[1][rest], good[1][rest])
    assert torch.isnan(y[1]).all() and torch.isfinite(y[rest].float()).all()
    if H % 128 == 0:
        _, _, c, s = moe.norm(x, None, 1e-6, q_mode=moe.Q_FP8_G128_POW2)
        torch.cuda.synchronize()
        # NaN spreads over its row; an infinite row is 0 but for 0 * inf in its own place
        want = torch.zeros_like(s, dtype=torch.bool)
        want[1], want[2, (H - 1) // 128], want[3, 0] = True, True, True
        assert torch.equal(s == 255, want)
        assert not c.view(T, H // 128, 128)[want].any()


# ---------------------------------------------------------------- quant_rows
@pytest.mark.parametrize("T,H,shift", [(1, 1, 0), (3, 16, 0), (32, 768, 0), (1023, 512, 0), (1024, 512, 0),
                                       (2050, 2048, 0), (4, 16384, 0), (5, 1111, 0), (3, 16383, 0), (6, 512, 3)])
def test_quant_rows(gpu, T, H, shift):
    import torch
    r = _rng(T, H, shift, 9)
    x = _bf16(_rows_values(r, T, H), gpu, shift)
    _say(f"[quant] T={T} H={H} shift={shift}")
    codes, scales = moe.quant_rows(x)
    torch.cuda.synchronize()
    _check_codes_i8(codes, scales, _f64(x), 127 * 3 * U, 2 * U)


def test_quant_rows_of_largest_and_smallest_values(gpu):
    import torch
    x = np.zeros((4, 64))
    x[0, 5] = 3.38e38
    x[1, 7], x[1, 8] = 2.0 ** -100, -(2.0 ** -101)
    x[2, 0] = 2.0 ** -126
    x = _bf16(x, gpu)
    codes, scales = moe.quant_rows(x)
    torch.cuda.synchronize()
    _check_codes_i8(codes, scales, _f64(x), 127 * 3 * U, 2 * U)
    assert int(codes[0, 5]) == 127 and int(codes[1, 7]) == 127 and not codes[3].any()


# ---------------------------------------------------------------- products
def _operands(r, M, N, K, full=False):
    lo, hi = (-128, 128)
    if full:                                            # the extremes only: the largest sums
        a, b = np.where(r.random((M, K)) < 0.9, -128, 127), np.where(r.random((N, K)) < 0.9, -128, 127)
    else:
        a, b = r.integers(lo, hi, (M, K)), r.integers(lo, hi, (N, K))
    sa = 0.028 * np.exp(0.3 * r.normal(size=M))
    sb = 0.028 / np.sqrt(K) * np.exp(0.3 * r.normal(size=N))
    return a, sa, b, sb


def _gemm_case(gpu, M, N, K, bias, add, f32, full=False, key=0):
    import torch
    r = _rng(M, N, K, bias, add, f32, key)
    _say(f"[gemm] M={M} N={N} K={K} bias={bias} add={add} f32={f32}")
    a, sa, b, sb = _operands(r, M, N, K, full)
    da, db, dsa, dsb = _i8(a, gpu), _i8(b, gpu), _f32(sa, gpu), _f32(sb, gpu)
    ot = torch.float32 if f32 else torch.bfloat16
    dbias = _f32(r.normal(size=N), gpu) if bias else None
    dadd = _f32(r.normal(size=(M, N)), gpu).to(ot) if add else None
    out = moe.gemm_i8(da, dsa, db, dsb, bias=dbias, add=dadd, out_dtype=ot)
    torch.cuda.synchronize()
    b64 = None if dbias is None else _f64(dbias)
    a64 = None if dadd is None else _f64(dadd)
    p, ref = dense.gemm_i8(a, _f64(dsa), b, _f64(dsb), b64, a64)
    mag = np.abs(p) + (0 if b64 is None else np.abs(b64)[None, :]) + (0 if a64 is None else np.abs(a64))
    _close("out", _f64(out), ref, 4 * U * mag + (0 if f32 else HB * np.abs(ref)) + 2.0 ** -133)


GEMM_SHAPES = [(1, 1, 16), (1, 2048, 2048), (2, 7, 48), (15, 16, 64), (16, 17, 80), (17, 33, 112), (31, 128, 128),
               (32, 2048, 512), (33, 64, 144), (48, 200, 1024), (63, 31, 256), (64, 512, 768), (65, 513, 272),
               (100, 1000, 4112), (128, 256, 2048), (129, 255, 400), (200, 2048, 512), (255, 257, 2064),
               (256, 512, 128), (257, 100, 16), (333, 1000, 1040), (520, 640, 896), (1024, 2048, 256), (1031, 999, 640),
               (2300, 2048, 384), (4100, 1100, 160)]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm_i8(gpu, M, N, K):
    _gemm_case(gpu, M, N, K, False, False, False)
    _gemm_case(gpu, M, N, K, True, True, True)


@pytest.mark.parametrize("M,N,K", [(1, 9, 64), (20, 130, 192), (70, 515, 320), (300, 2048, 512), (1100, 513, 144)])
@pytest.mark.parametrize("bias,add,f32", [(True, False, False), (False, True, False), (True, True, False),
                                          (False, False, True)])
def test_gemm_i8_epilogues(gpu, M, N, K, bias, add, f32):
    _gemm_case(gpu, M, N, K, bias, add, f32)


@pytest.mark.parametrize("M,N", [(3, 40), (40, 70), (300, 260)])
def test_gemm_i8_largest_sums(gpu, M, N):
    """K at its limit with codes at the ends of their range: sums up to 2^31 - 2^18."""
    _gemm_case(gpu, M, N, 131056, False, False, True, full=True)


@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (24, 520, 512), (80, 512, 1024), (300, 1000, 384), (1200, 2048, 256)])
def test_gemm_i8_adds_in_place(gpu, M, N, K):
    import torch
    r = _rng(M, N, K, 21)
    a, sa, b, sb = _operands(r, M, N, K)
    args = (_i8(a, gpu), _f32(sa, gpu), _i8(b, gpu), _f32(sb, gpu))
    base = _bf16(r.normal(size=(M, N)), gpu)
    want = moe.gemm_i8(*args, add=base)
    got = base.clone()
    assert moe.gemm_i8(*args, add=got, out=got) is got
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_gemm_i8_unaligned_output(gpu):
    import torch
    r = _rng(22)
    for M, N, K in ((5, 64, 128), (300, 512, 256)):
        a, sa, b, sb = _operands(r, M, N, K)
        args = (_i8(a, gpu), _f32(sa, gpu), _i8(b, gpu), _f32(sb, gpu))
        want = moe.gemm_i8(*args)
        buf = torch.full((M * N + 8,), 7.0, dtype=torch.bfloat16, device=gpu)
        out = buf[1:1 + M * N].view(M, N)
        moe.gemm_i8(*args, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert (buf[0] == 7) and (buf[1 + M * N:] == 7).all()


def test_products_write_nothing_past_their_rows(gpu):
    import torch
    r = _rng(23)
    for M, N, K in ((1, 17, 64), (33, 65, 128), (257, 300, 256), (1030, 264, 128)):
        a, sa, b, sb = _operands(r, M, 2 * N, K)
        args = (_i8(a, gpu), _f32(sa, gpu), _i8(b, gpu), _f32(sb, gpu))
        for n, f in ((2 * N, moe.gemm_i8), (N, moe.glu_i8)):
            buf = torch.full((M * n + 512,), 7.0, dtype=torch.bfloat16, device=gpu)
            f(*args, out=buf[:M * n].view(M, n))
            torch.cuda.synchronize()
            assert (buf[M * n:] == 7).all()


def test_nan_scales_stay_in_their_rows(gpu):
    """A row whose int8 scale is NaN (a non-finite token) gives a NaN row, and no other."""
    import torch
    r = _rng(24)
    for M in (8, 40, 300):
        a, sa, b, sb = _operands(r, M, 256, 256)
        sa[M // 2] = np.nan
        args = (_i8(a, gpu), _f32(sa, gpu), _i8(b, gpu), _f32(sb, gpu))
        for o in (moe.gemm_i8(*args), moe.glu_i8(*args)):
            torch.cuda.synchronize()
            bad = torch.isnan(o).all(dim=1)
            assert bad[M // 2] and int(bad.sum()) == 1 and int(torch.isnan(o).any(dim=1).sum()) == 1


def _glu_case(gpu, M, I, K, gain=1.0, key=0):
    import torch
    r = _rng(M, I, K, 31, key)
    _say(f"[glu] M={M} I={I} K={K} gain={gain}")
    a, sa, b, sb = _operands(r, M, 2 * I, K)
    da, db, dsa, dsb = _i8(a, gpu), _i8(b, gpu), _f32(sa * gain, gpu), _f32(sb, gpu)
    out = moe.glu_i8(da, dsa, db, dsb)
    torch.cuda.synchronize()
    g, u, ref = dense.glu_i8(a, _f64(dsa), b, _f64(dsb))
    tol = np.abs(ref) * (HB + (4 * np.abs(g) + 16) * U) + 2.0 ** -125 * np.abs(g * u) + 2.0 ** -133
    _close("h", _f64(out), ref, tol)


@pytest.mark.parametrize("M,I,K", [(1, 1, 16), (1, 512, 2048), (2, 7, 48), (8, 512, 2048), (16, 9, 64), (17, 768, 272),
                                   (32, 100, 512), (33, 64, 128), (64, 512, 768), (65, 513, 144), (128, 128, 2048),
                                   (129, 257, 400), (256, 512, 128), (257, 50, 16), (333, 500, 1040), (600, 768, 640),
                                   (1031, 333, 320), (2300, 512, 256), (4100, 520, 160)])
def test_glu_i8(gpu, M, I, K):
    _glu_case(gpu, M, I, K)


@pytest.mark.parametrize("M", [5, 50, 400])
def test_glu_i8_wide_gates(gpu, M):
    """Gates far past where the exponential over- and underflows."""
    _glu_case(gpu, M, 192, 512, gain=60.0)


@pytest.mark.parametrize("M", [5, 50, 400])
def test_glu_i8_closed_gates_of_huge_products(gpu, M):
    """g far below zero with g u past fp32: silu(g) is 0 there, and so is h."""
    import torch
    a = _i8(np.full((M, 64), 127), gpu)
    w = _i8(np.concatenate([np.full((40, 64), -127), np.full((40, 64), 127)]), gpu)
    h = moe.glu_i8(a, torch.full((M,), 1e8, device=gpu), w, torch.full((80,), 1e8, device=gpu))
    torch.cuda.synchronize()
    assert (h == 0).all()


def test_results_repeat_bit_for_bit(gpu):
    import torch
    r = _rng(25)
    for M, N, K in ((4, 2048, 4096), (150, 1000, 8192), (700, 512, 2048)):
        a, sa, b, sb = _operands(r, M, N, K)
        args = (_i8(a, gpu), _f32(sa, gpu), _i8(b, gpu), _f32(sb, gpu))
        for f in (moe.gemm_i8, moe.glu_i8):
            o = [f(*args) for _ in range(3)]
            torch.cuda.synchronize()
            assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2])


# ---------------------------------------------------------------- together
def _block(T, H, I, dev, key=0):
    r = _rng(T, H, I, 41, key)
    x, rs = (_bf16(r.normal(size=(T, H)), dev) for _ in range(2))
    w = _f32(1 + 0.2 * r.normal(size=H), dev)
    w13, w2 = _i8(r.integers(-127, 128, (2 * I, H)), dev), _i8(r.integers(-127, 128, (H, I)), dev)
    s13, s2 = (_f32(0.02 / 73 * np.exp(0.2 * r.normal(size=n)), dev) for n in (2 * I, H))
    routed = _bf16(r.normal(size=(T, H)), dev)
    return x, rs, w, w13, s13, w2, s2, routed


def _run_block(x, rs, w, w13, s13, w2, s2, routed, **k):
    y, total, q, sc = moe.norm(x, w, 1e-6, res=rs, q_mode=moe.Q_I8_ROW, **k)
    return y, total, moe.shared_expert_i8(q, sc, w13, s13, w2, s2, add=routed, **k)


@pytest.mark.parametrize("T,H,I", [(1, 2048, 512), (8, 2048, 768), (50, 512, 256), (300, 2048, 512), (1500, 1024, 768)])
def test_shared_expert_chain(gpu, T, H, I):
    """norm -> gated product -> row quantizer -> product + the routed experts'
    output: each step against the oracle on what the step before wrote."""
    import torch
    x, rs, w, w13, s13, w2, s2, routed = _block(T, H, I, gpu)
    _say(f"[chain] T={T} H={H} I={I}")
    y, total, out = _run_block(x, rs, w, w13, s13, w2, s2, routed)
    _, _, q, sc = moe.norm(x, w, 1e-6, res=rs, q_mode=moe.Q_I8_ROW)
    h = moe.glu_i8(q, sc, w13, s13)
    hq, hs = moe.quant_rows(h)
    torch.cuda.synchronize()
    ry, _ = dense.rms_norm(_f64(x), _f64(w), 1e-6, _f64(rs))
    _check_codes_i8(q, sc, ry, 1e-3, 66 * U)
    g, u, rh = dense.glu_i8(q.cpu().numpy(), _f64(sc), w13.cpu().numpy(), _f64(s13))
    _close("h", _f64(h), rh, np.abs(rh) * (HB + (4 * np.abs(g) + 16) * U) + 2.0 ** -133)
    _check_codes_i8(hq, hs, _f64(h), 127 * 3 * U, 2 * U)
    p, ro = dense.gemm_i8(hq.cpu().numpy(), _f64(hs), w2.cpu().numpy(), _f64(s2), None, _f64(routed))
    _close("out", _f64(out), ro, 4 * U * (np.abs(p) + np.abs(_f64(routed))) + HB * np.abs(ro) + 2.0 ** -133)


def test_norm_feeds_the_expert_layer(gpu):
    """The norm's rows through the router gate and the expert layer, the shared
    expert added to the layer's output: the fused steps give what the separate
    calls give."""
    import torch
    from gen import CONFIGS, make_layer, make_bank, router_inputs
    from harness import device_pool, device_inputs, oracle_layer, rel_max_err
    c = CONFIGS["C0"]
    li = make_layer(c, 16, 3)
    bank = make_bank(c)
    pool = device_pool(li, bank, gpu)
    x, _, soe, mask = device_inputs(li, gpu)
    _, rs, w, w13, s13, w2, s2, _ = _block(16, c.H, c.I, gpu)
    y, total, q, sc = moe.norm(x, w, 1e-6, res=rs, q_mode=moe.Q_I8_ROW)
    Wg = _f32(router_inputs(c, 16, 3)[0], gpu)
    logits, ids, tw, err = moe.route_gemm(y, Wg, c.k)
    routed, (ids2, _, _), _ = moe.layer(pool, y, logits, c.k, soe, 16, moe.ACT_BF16, mask=mask, fused="layer")
    out = moe.shared_expert_i8(q, sc, w13, s13, w2, s2, add=routed)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2)
    li2 = type(li)(**{**li.__dict__, "logits": logits.cpu().numpy(),
                      "x_bits": y.view(torch.int16).cpu().numpy().view(np.uint16)})
    ref = oracle_layer(li2, bank, 16, moe.ACT_BF16)
    assert rel_max_err(routed, ref["out"]) <= 2e-2
    hq, hs = moe.quant_rows(moe.glu_i8(q, sc, w13, s13))
    torch.cuda.synchronize()
    p, ro = dense.gemm_i8(hq.cpu().numpy(), _f64(hs), w2.cpu().numpy(), _f64(s2), None, _f64(routed))
    _close("out", _f64(out), ro, 4 * U * (np.abs(p) + np.abs(_f64(routed))) + HB * np.abs(ro) + 2.0 ** -133)


@pytest.mark.parametrize("T,H,I", [(2, 2048, 512), (64, 1024, 512), (300, 512, 256)])
def test_chain_on_another_stream_and_in_a_graph(gpu, T, H, I):
    import torch
    args = _block(T, H, I, gpu, 1)
    want = [t.clone() for t in _run_block(*args)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _run_block(*args, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _run_block(*args)
    other = _block(T, H, I, gpu, 2)
    for k in range(4):                                  # new inputs in the captured tensors, eager work between replays
        src = args if k % 2 else other
        fresh = [t.clone() for t in src[:2]]
        keep = [args[0].clone(), args[1].clone()]
        args[0].copy_(fresh[0])
        args[1].copy_(fresh[1])
        eager = [t.clone() for t in _run_block(*args)]
        for t in held:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b), k
        args[0].copy_(keep[0])
        args[1].copy_(keep[1])


def test_two_streams_at_once(gpu):
    """Two chains in flight together share nothing."""
    import torch
    A, B = _block(200, 1024, 512, gpu, 5), _block(40, 2048, 256, gpu, 6)
    wa, wb = _run_block(*A), _run_block(*B)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for k in range(6):
        outs.append((_run_block(*(A, B)[k % 2], stream=s[k % 2]), (wa, wb)[k % 2]))
    torch.cuda.synchronize()
    for got, want in outs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_refusals_on_the_device(gpu):
    import torch
    a = torch.zeros(4, 64, dtype=torch.int8, device=gpu)
    s = torch.ones(4, device=gpu)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=gpu)
    bad = [lambda: moe.gemm_i8(a, s, a[:, :48], s),                               # not contiguous
           lambda: moe.gemm_i8(a, s, a[:, :48].contiguous(), s),                  # another K
           lambda: moe.gemm_i8(a, s[:3], a, s), lambda: moe.gemm_i8(a, s, a, s, bias=s[:2]),
           lambda: moe.gemm_i8(a, s, a, s, add=torch.zeros(4, 4, device=gpu)),    # add's type is not out's
           lambda: moe.gemm_i8(a, s, a, s, out_dtype=torch.float16),
           lambda: moe.gemm_i8(a.to(torch.uint8), s, a, s), lambda: moe.gemm_i8(a, s.cpu(), a, s),
           lambda: moe.gemm_i8(a[:, :8].contiguous(), s, a[:, :8].contiguous(), s),   # K = 8
           lambda: moe.glu_i8(a, s, a[:3], s[:3]), lambda: moe.glu_i8(a, s, a, s[:2]),
           lambda: moe.norm(x.float()), lambda: moe.norm(x, s), lambda: moe.norm(x, with_y=False),
           lambda: moe.norm(x, res=x[:2]), lambda: moe.norm(x, q_mode=5), lambda: moe.norm(x, eps=0.0),
           lambda: moe.norm(x, q_mode=moe.Q_FP8_G128_POW2), lambda: moe.quant_rows(x.t()),
           lambda: moe.quant_rows(torch.zeros(1, 16385, dtype=torch.bfloat16, device=gpu))]
    for k, call in enumerate(bad):
        with pytest.raises(moe.MoeError):
            call()
            _say("not refused:", k)


@pytest.mark.parametrize("M,N,K", [(4100, 1101, 160), (2300, 2047, 384), (700, 1023, 208), (90, 259, 144), (5000, 5, 64), (3000, 1030, 96)])
def test_products_of_rows_that_start_anywhere(gpu, M, N, K):
    """Odd row lengths (any start of a row, lanes that end inside one) in every tile size, with and without addend."""
    import torch
    for bias, add, f32 in ((False, False, False), (True, True, False), (False, True, True)):
        _gemm_case(gpu, M, N, K, bias, add, f32, key=9)
    _glu_case(gpu, M, N, K)
    r = _rng(M, N, K, 31)
    a, sa, b, sb = _operands(r, M, N, K)
    args = (_i8(a, gpu), _f32(sa, gpu), _i8(b, gpu), _f32(sb, gpu))
    for t, shift in ((torch.bfloat16, 1), (torch.bfloat16, 4), (torch.float32, 1)):
        want = moe.gemm_i8(*args, out_dtype=t)
        buf = torch.full((M * N + 64,), 7.0, dtype=t, device=gpu)
        moe.gemm_i8(*args, out=buf[shift:shift + M * N].view(M, N))
        torch.cuda.synchronize()
        assert torch.equal(buf[shift:shift + M * N].view(M, N), want)
        assert (buf[:shift] == 7).all() and (buf[shift + M * N:] == 7).all()
