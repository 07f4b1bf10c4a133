"""8-bit rows of the dense operators: codes that are exactly the definition's,
rows on every alignment, and the way back to bf16.

Row arithmetic is fp64 behind an fp32 sum x + res, so a code can differ from
the fp64 oracle's only where its argument lies within some 2^-45 of a border:
with the fixed inputs here none does (the oracle's own distance from the
borders is checked), and codes have to be equal, not near.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import dense, e4m3_decode
from test_gpu_dense import HB, U, _bf16, _close, _f32, _f64, _rng, _rows_values, _say

pytestmark = pytest.mark.gpu


def _i8_exact(name, codes, t):
    c = codes.cpu().numpy().astype(np.int64)
    want = np.rint(t).astype(np.int64)
    far = np.abs(np.abs(t - np.floor(t)) - 0.5) > 2.0 ** -40          # not within rounding of a border
    _say(f"    {name}: {int((~far).sum())} of {t.size} on a border, {int((c != want).sum())} differ")
    assert np.array_equal(c[far], want[far])


@pytest.mark.parametrize("T,H", [(1, 1), (2, 5), (3, 9), (1025, 9), (1030, 63), (1027, 511), (1100, 1023), (1024, 2041),
                                 (1025, 2047), (9, 2049), (5, 4095), (7, 8191), (3, 16377), (3, 16381), (40, 333), (2000, 2048)])
def test_norm_codes_are_exact(gpu, T, H):
    import torch
    r = _rng(T, H, 51)
    x, rs = (_bf16(_rows_values(r, T, H), gpu) for _ in range(2))
    w = _f32(1 + 0.2 * r.normal(size=H), gpu)
    _say(f"[norm codes] T={T} H={H}")
    y, total, codes, scales = moe.norm(x, w, 1e-6, res=rs, q_mode=moe.Q_I8_ROW)
    torch.cuda.synchronize()
    v = (x.float() + rs.float()).double().cpu().numpy()               # the fp32 sum the kernel takes
    ry, _ = dense.rms_norm(v, _f64(w), float(np.float32(1e-6)))
    t, s = dense.i8_rows(ry)
    _i8_exact("codes", codes, t)
    _close("scales", _f64(scales), s, s * 2 * U)
    _close("y", _f64(y), ry, np.abs(ry) * (HB + 2 * U) + 2.0 ** -133)
    _close("sum", _f64(total), v, np.abs(v) * HB + 2.0 ** -133)


@pytest.mark.parametrize("T,H", [(1, 128), (70, 256), (1100, 512), (6, 16384), (1500, 2048)])
def test_norm_e4m3_codes_are_exact(gpu, T, H):
    import torch
    r = _rng(T, H, 52)
    x, rs = (_bf16(_rows_values(r, T, H), gpu) for _ in range(2))
    _, _, codes, scales = moe.norm(x, None, 1e-6, res=rs, q_mode=moe.Q_FP8_G128_POW2)
    torch.cuda.synchronize()
    ry, _ = dense.rms_norm((x.float() + rs.float()).double().cpu().numpy(), None, float(np.float32(1e-6)))
    g = ry.reshape(T, H // 128, 128)
    m = np.abs(g).max(axis=2)
    e = np.where(m > 0, np.ceil(np.log2(np.where(m > 0, m, 1.0) / 448)), 0).astype(np.int64)
    assert np.array_equal(scales.cpu().numpy().astype(np.int64) - 127, e)
    z = g / np.exp2(e)[:, :, None]
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -20))), -6) - 3)
    assert np.array_equal(e4m3_decode(codes.cpu().numpy()).reshape(z.shape), np.rint(z / step) * step)


def _exact_rint(x, m):
    """rint(127 x / m) of bf16 rows, ties to even, in integers: x = X 2^-k, m = Mx 2^-k exactly."""
    k = 140
    X = np.array([[int(v) for v in row] for row in np.ldexp(x, k).astype(object)], dtype=object)
    out = np.empty(x.shape, dtype=np.int64)
    for i in range(x.shape[0]):
        d = int(np.ldexp(float(m[i]), k))
        for j in range(x.shape[1]):
            q, rem = divmod(2 * 127 * X[i, j] + d, 2 * d)             # floor(127 x / m + 1/2)
            out[i, j] = q - 1 if rem == 0 and q % 2 else q
    return out


@pytest.mark.parametrize("H", [64, 333, 2048])
def test_quant_rows_codes_are_exact_with_ties(gpu, H):
    """Rows whose largest value is a small integer times a power of two: 127 x / m falls on borders."""
    import torch
    r = _rng(H, 53)
    T = 12
    x = r.integers(-255, 256, (T, H)) * np.exp2(r.integers(-4, 4, (T, 1)))
    for i, top in enumerate((256, 254, 508, 2, 4, 256, 384, 320, 254, 255, 256, 512)):
        x[i] = np.clip(x[i], -top, top)
        x[i, 3 % H] = top
    xb = _bf16(x, gpu)
    codes, scales = moe.quant_rows(xb)
    torch.cuda.synchronize()
    v = _f64(xb)
    m = np.abs(v).max(axis=1)
    want = _exact_rint(v, m)
    t = 127 * v / m[:, None]
    _say(f"    ties {int((np.abs(t - np.floor(t)) == 0.5).sum())}")
    assert np.array_equal(codes.cpu().numpy().astype(np.int64), want)
    _close("scales", _f64(scales), m / 127, m / 127 * 2 * U)


@pytest.mark.parametrize("T,H", [(1030, 9), (3, 1111), (2, 2047), (1500, 333)])
def test_shifted_rows_write_only_their_own(gpu, T, H):
    """Odd rows: what lies behind each output stays as it was, and each row's bytes are its own."""
    import torch
    r = _rng(T, H, 54)
    x, rs = (_bf16(_rows_values(r, T, H), gpu) for _ in range(2))
    n = T * H
    yb, sb = (torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    cb, fb = torch.full((n + 64,), 55, dtype=torch.int8, device=gpu), torch.full((T + 16,), 7.0, device=gpu)
    moe.norm(x, None, 1e-6, res=rs, q_mode=moe.Q_I8_ROW, y=yb[:n].view(T, H), sum=sb[:n].view(T, H),
             codes=cb[:n].view(T, H), scales=fb[:T])
    one = [moe.norm(x[i:i + 1].clone(), None, 1e-6, res=rs[i:i + 1].clone(), q_mode=moe.Q_I8_ROW) for i in (0, 1, T // 2, T - 1)]
    torch.cuda.synchronize()
    assert (yb[n:] == 7).all() and (sb[n:] == 7).all() and (cb[n:] == 55).all() and (fb[T:] == 7).all()
    for i, (y, s, c, f) in zip((0, 1, T // 2, T - 1), one):
        assert torch.equal(yb[:n].view(T, H)[i], y[0]) and torch.equal(sb[:n].view(T, H)[i], s[0])
        assert torch.equal(cb[:n].view(T, H)[i], c[0]) and torch.equal(fb[i], f[0])


@pytest.mark.parametrize("T,H,shift", [(1, 1, 0), (3, 7, 0), (5, 64, 0), (40, 1000, 0), (1100, 2048, 0), (6, 64, 1)])
def test_dequant_rows(gpu, T, H, shift):
    import torch
    r = _rng(T, H, shift, 55)
    buf = torch.from_numpy(r.integers(-128, 128, T * H + shift).astype(np.int8)).to(gpu)
    codes = buf[shift:].view(T, H)
    scales = _f32(np.exp(r.normal(size=T)), gpu)
    if T > 2:
        scales[1] = float("nan")
    out = torch.full((T * H + 8,), 7.0, dtype=torch.bfloat16, device=gpu)
    moe.dequant_rows(codes, scales, out=out[:T * H].view(T, H))
    torch.cuda.synchronize()
    got = _f64(out[:T * H].view(T, H))
    ref = codes.cpu().numpy().astype(np.float64) * _f64(scales)[:, None]
    keep = ~np.isnan(ref).any(axis=1)
    assert np.isnan(got[~keep]).all() and (out[T * H:] == 7).all()
    _close("values", got[keep], ref[keep], np.abs(ref[keep]) * (HB + U) + 2.0 ** -133)


def test_dequant_rows_e4m3(gpu):
    import torch
    x = _bf16(_rows_values(_rng(56), 50, 384), gpu)
    codes, exps = moe.quant_act(x)
    exps[3, 1] = 255
    out = moe.dequant_rows(codes, exps)
    torch.cuda.synchronize()
    e = exps.cpu().numpy().astype(np.float64) - 127
    ref = (e4m3_decode(codes.cpu().numpy()).reshape(50, 3, 128) * np.exp2(e)[:, :, None])
    got = _f64(out).reshape(50, 3, 128)
    assert np.isnan(got[3, 1]).all()
    got[3, 1] = ref[3, 1] = 0
    assert np.array_equal(got, ref)                                   # e4m3 times a power of two fits bf16


def test_norm_of_rows_past_fp32(gpu):
    """Values whose squares overflow fp32, and rows far below it: the fp64 sum holds both."""
    import torch
    r = _rng(57)
    x = r.normal(size=(4, 300))
    x[0] *= 1e37
    x[1] *= 1e30
    x[2] *= 1e-30
    xb = _bf16(x, gpu)
    y, _, codes, scales = moe.norm(xb, None, 1e-6, q_mode=moe.Q_I8_ROW)
    torch.cuda.synchronize()
    ry, _ = dense.rms_norm(_f64(xb), None, float(np.float32(1e-6)))
    _close("y", _f64(y), ry, np.abs(ry) * (HB + 2 * U) + 2.0 ** -133)
    t, s = dense.i8_rows(ry)
    _i8_exact("codes", codes, t)


def test_dequant_refusals(gpu):
    import torch
    c = torch.zeros(4, 64, dtype=torch.int8, device=gpu)
    for call in (lambda: moe.dequant_rows(c, torch.zeros(3, device=gpu)),
                 lambda: moe.dequant_rows(c.view(torch.uint8), torch.zeros(4, 1, dtype=torch.uint8, device=gpu)),
                 lambda: moe.dequant_rows(c.float(), torch.zeros(4, device=gpu)),
                 lambda: moe.dequant_rows(c.t(), torch.zeros(64, device=gpu))):
        with pytest.raises(moe.MoeError):
            call()


def test_norm_refuses_a_y_that_it_would_not_write(gpu):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=gpu)
    with pytest.raises(moe.MoeError):
        moe.norm(x, res=x, with_y=False, y=torch.empty_like(x))


@pytest.mark.parametrize("T,H", [(2049, 1032), (2050, 2047), (2100, 2048), (2060, 1025)])
def test_norm_codes_are_exact_in_many_long_rows(gpu, T, H):
    """From 2049 rows on a wave takes rows of more than 1024 columns too."""
    test_norm_codes_are_exact(gpu, T, H)
    if H % 128 == 0:
        test_norm_e4m3_codes_are_exact(gpu, T, H)


@pytest.mark.parametrize("T,H", [(1, 1), (9, 1), (40, 2), (33, 7), (70, 9), (1001, 333), (5, 4099)])
@pytest.mark.parametrize("shift", [0, 1])
def test_dequant_rows_of_any_length(gpu, T, H, shift):
    """Eight values at a time over rows of any length: several rows in one vector, a tensor that ends inside one."""
    import torch
    r = _rng(T, H, 61)
    buf = torch.zeros(T * H + shift, dtype=torch.int8, device=gpu)
    codes = buf[shift:].view(T, H)
    codes.copy_(torch.from_numpy(r.integers(-128, 128, (T, H)).astype(np.int8)))
    scales = _f32(np.exp(r.normal(size=T)), gpu)
    guard = torch.full((T * H + 64,), 7.0, dtype=torch.bfloat16, device=gpu)
    out = moe.dequant_rows(codes, scales, out=guard[:T * H].view(T, H))
    torch.cuda.synchronize()
    want = (codes.float() * scales[:, None]).to(torch.bfloat16)      # one product, one rounding: the same bits
    assert torch.equal(out, want) and (guard[T * H:] == 7).all()
