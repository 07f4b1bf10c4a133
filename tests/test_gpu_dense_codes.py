"""8-bit rows of the norm and the quantizer where a code is hardest to decide:
arguments next to a border, weights, every output mode and kernel form.

Tolerances: v = x + res is one fp32 rounding, and the reference takes it from
there; sums, r and y are fp64 (relative errors of some 2^-50), so a code is the
definition's wherever its argument is 2^-40 and more away from a border, and a
bf16 output is two roundings away from y, to fp32 and to bf16: 2^-24 + 2^-8 of
it, or 2^-134 below bf16's normal values (half a step).
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import dense, e4m3_decode
from test_gpu_dense import HB, U, _bf16, _close, _f32, _f64, _rng, _rows_values, _say
from test_gpu_dense_rows import _exact_rint, _i8_exact

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _e4m3_exact(codes, scales, y):
    """e4m3 codes and E8M0 bytes against the definition of the unrounded y."""
    T, H = y.shape
    g = y.reshape(T, H // 128, 128)
    m = np.abs(g).max(axis=2)
    e = np.where(m > 0, np.ceil(np.log2(np.where(m > 0, m, 1.0) / 448)), 0).clip(-127, 127).astype(np.int64)
    assert np.array_equal(scales.cpu().numpy().astype(np.int64) - 127, e)
    z = g / np.exp2(e.astype(np.float64))[:, :, None]
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -20))), -6) - 3)
    t = z / step
    far = np.abs(np.abs(t - np.floor(t)) - 0.5) > 2.0 ** -40
    c = e4m3_decode(codes.cpu().numpy()).reshape(z.shape)
    want = np.rint(t) * step
    _say(f"    e4m3: {int((~far).sum())} of {t.size} on a border, {int((c != want)[far].sum())} differ")
    assert np.array_equal(c[far], want[far])


@pytest.mark.parametrize("T", [12, 1100])
def test_quant_rows_next_to_every_kind_of_border(gpu, T):
    """The bf16 pairs (x, m) whose 127 x / m lies closest to a border without
    being on it, for each distance in binades (down to 1 / 64768: 255 2^-8 under
    253), beside pairs that are on one."""
    import torch
    pairs = []
    for j in range(9):
        near = []
        for X in range(128, 256):
            for M in range(128, 256):
                if j == 0 and X > M:
                    continue
                d = M << j
                off = abs((254 * X) % (2 * d) - d)                    # |2 t - nearest odd number| in units of 1 / d
                near.append((off / d, X, M, j))
        near.sort()
        pairs += [p[1:] for p in near if p[0] > 0][:24] + [p[1:] for p in near if p[0] == 0][:8]
    x = np.zeros((len(pairs), 2 * len(pairs)))
    for i, (X, M, j) in enumerate(pairs):
        x[i, 0] = M
        x[i, 1:len(pairs)] = X * 2.0 ** -j
        x[i, len(pairs):] = -X * 2.0 ** -j
    x *= np.exp2(np.arange(len(pairs)) % 60 - 30)[:, None]
    if T > len(pairs):
        x = np.concatenate([x] * (T // len(pairs) + 1))
    xb = _bf16(x, gpu)
    codes, scales = moe.quant_rows(xb)
    torch.cuda.synchronize()
    v = _f64(xb)
    assert np.array_equal(v, x)
    c = codes.cpu().numpy().astype(np.int64)
    for lo in range(0, len(x), len(pairs)):                           # (the rows repeat)
        assert np.array_equal(c[lo:lo + len(pairs)], c[:len(pairs)])
    cols = [0, 1, 2, len(pairs) - 1, len(pairs), 2 * len(pairs) - 1]
    want = _exact_rint(v[:len(pairs)][:, cols], np.abs(v[:len(pairs)]).max(axis=1))
    assert np.array_equal(c[:len(pairs)][:, cols], want)
    assert np.array_equal(c[:len(pairs), 1:len(pairs)], np.repeat(want[:, 1:2], len(pairs) - 1, axis=1))
    assert np.array_equal(c[:len(pairs), len(pairs):], np.repeat(want[:, 4:5], len(pairs), axis=1))


@pytest.mark.parametrize("T,H,shift", [(1, 128, 0), (70, 256, 0), (1100, 512, 0), (6, 16384, 0), (2100, 2048, 0), (5, 4096, 0),
                                       (3, 7, 0), (1030, 333, 0), (9, 4099, 0), (9, 512, 1), (4, 2176, 4)])
@pytest.mark.parametrize("res,w", [(True, True), (True, False), (False, True), (False, False)])
def test_norm_in_every_mode(gpu, T, H, shift, res, w):
    import torch
    r = _rng(T, H, shift, res, w, 81)
    x = _bf16(_rows_values(r, T, H), gpu, shift)
    rs = _bf16(_rows_values(r, T, H), gpu, shift) if res else None
    wt = _f32(1 + 0.2 * r.normal(size=H), gpu) if w else None
    v = x.float() + rs.float() if res else x.float()
    v64 = v.double().cpu().numpy()
    ry, _ = dense.rms_norm(v64, None if wt is None else _f64(wt), float(np.float32(EPS)))
    modes = [moe.Q_NONE, moe.Q_I8_ROW] + ([moe.Q_FP8_G128_POW2] if H % 128 == 0 and not shift else [])
    for q in modes:
        _say(f"[norm] T={T} H={H} shift={shift} res={res} w={w} q={q}")
        y, total, codes, scales = moe.norm(x, wt, EPS, res=rs, q_mode=q)
        torch.cuda.synchronize()
        _close("y", _f64(y), ry, np.abs(ry) * (HB + U + 2.0 ** -40) + 2.0 ** -134)
        if res:
            assert torch.equal(total, v.to(torch.bfloat16))
        if q == moe.Q_I8_ROW:
            t, s = dense.i8_rows(ry)
            _i8_exact("codes", codes, t)
            _close("scales", _f64(scales), s, s * (U + 2.0 ** -40))
        if q == moe.Q_FP8_G128_POW2:
            _e4m3_exact(codes, scales, ry)


@pytest.mark.parametrize("T,H,shift", [(40, 512, 0), (1100, 256, 0), (1030, 333, 0), (2100, 1032, 0), (9, 512, 1), (5, 4099, 0)])
@pytest.mark.parametrize("res,w", [(False, False), (True, False), (False, True)])
def test_norm_codes_with_ties(gpu, T, H, shift, res, w):
    """127 y / m does not depend on r, so rows of small integers have it exactly
    on a border (with weights that are powers of two as well): ties go to the
    even code, decided here in integers."""
    import torch
    r = _rng(T, H, shift, res, w, 82)
    x = r.integers(-255, 256, (T, H)).astype(np.float64)
    tops = np.array([256, 254, 508, 2, 4, 384, 320, 255, 512, 380])[np.arange(T) % 10]
    x = np.clip(x, -tops[:, None], tops[:, None])
    x[np.arange(T), np.arange(T) % H] = tops
    x *= np.exp2(r.integers(-20, 20, (T, 1)))
    xb = _bf16(x, gpu, shift)
    rs = _bf16(-0.5 * x, gpu, shift) if res else None                 # (the sum is x / 2)
    wt = np.full(H, 0.25) if w else None
    if w:
        wt[r.random(H) < 0.3] = 0.125
    v = x * (0.5 if res else 1.0)
    assert np.array_equal(_f64(xb), x)
    _, _, codes, _ = moe.norm(xb, None if wt is None else _f32(wt, gpu), EPS, res=rs, q_mode=moe.Q_I8_ROW)
    torch.cuda.synchronize()
    u = v * (1.0 if wt is None else wt[None, :])
    rows = np.unique(np.concatenate([np.arange(min(T, 20)), [T - 2, T - 1]]))
    want = _exact_rint(u[rows], np.abs(u[rows]).max(axis=1))
    t = 127 * u[rows] / np.abs(u[rows]).max(axis=1, keepdims=True)
    c = codes.cpu().numpy().astype(np.int64)[rows]
    _say(f"    ties {int((np.abs(t - np.floor(t)) == 0.5).sum())} of {t.size}, {int((c != want).sum())} differ")
    assert np.array_equal(c, want)


@pytest.mark.parametrize("T", [40, 1100])
@pytest.mark.parametrize("e", [-120, -124, -126, -128, -131])
def test_norm_e4m3_codes_of_tiny_rows(gpu, T, e):
    """y around 2^e: below 2^-126 fp32 holds fewer digits, and the scale stops at 2^-127."""
    import torch
    H = 1024
    r = _rng(T, -e, 83)
    x = _bf16(r.normal(size=(T, H)), gpu)
    w = _f32(2.0 ** e * (1 + r.integers(0, 64, H) / 64), gpu)         # (a few digits: fp32's subnormals hold them)
    _, _, codes, scales = moe.norm(x, w, EPS, q_mode=moe.Q_FP8_G128_POW2)
    torch.cuda.synchronize()
    ry, _ = dense.rms_norm(_f64(x), _f64(w), float(np.float32(EPS)))
    _e4m3_exact(codes, scales, ry)


@pytest.mark.parametrize("T", [5, 1100])
def test_norm_e4m3_codes_of_tiny_groups_beside_huge_ones(gpu, T):
    """Groups around 2^-124 and around 2^110 in one row, and in one wave."""
    import torch
    H = 1024
    r = _rng(T, 84)
    x = _bf16(r.normal(size=(T, H)), gpu)
    e = np.repeat(np.array([-124, 110, 110, -131, 0, -118, -124, 100]), 128)
    w = _f32(2.0 ** e * (1 + r.integers(0, 64, H) / 64), gpu)
    _, _, codes, scales = moe.norm(x, w, EPS, q_mode=moe.Q_FP8_G128_POW2)
    torch.cuda.synchronize()
    ry, _ = dense.rms_norm(_f64(x), _f64(w), float(np.float32(EPS)))
    _e4m3_exact(codes, scales, ry)


def test_inputs_that_require_a_gradient_are_read(gpu):
    """No operator has a gradient: outputs require none, and are what the plain tensors give."""
    import torch
    r = _rng(85)
    x = _bf16(r.normal(size=(5, 64)), gpu)
    w = _f32(1 + 0.1 * r.normal(size=64), gpu)
    b, sb = torch.zeros(16, 64, dtype=torch.int8, device=gpu) + 3, _f32(np.ones(16), gpu)
    plain = moe.norm(x, w, q_mode=moe.Q_I8_ROW)
    xg, wg, sg = x.clone().requires_grad_(), w.clone().requires_grad_(), sb.clone().requires_grad_()
    y, _, codes, scales = moe.norm(xg, wg, q_mode=moe.Q_I8_ROW)
    out = moe.gemm_i8(codes, scales, b, sg)
    torch.cuda.synchronize()
    assert not (y.requires_grad or scales.requires_grad or out.requires_grad)
    assert torch.equal(y, plain[0]) and torch.equal(codes, plain[2]) and torch.equal(scales, plain[3])
    assert torch.equal(out, moe.gemm_i8(plain[2], plain[3], b, sb))


@pytest.mark.parametrize("T,H,shift,q", [(5, 256, 0, 2), (1100, 512, 0, 2), (3, 4096, 0, 2), (7, 512, 1, 1), (1030, 333, 0, 1), (3, 4099, 3, 1),
                                         (9, 100, 5, 0)])
def test_norm_in_place_in_every_form(gpu, T, H, shift, q):
    """sum in x's memory and y in res's, and the other way round, on every kind of rows."""
    import torch
    r = _rng(T, H, shift, q, 86)
    x, rs = _bf16(_rows_values(r, T, H), gpu, shift), _bf16(_rows_values(r, T, H), gpu, shift)
    w = _f32(1 + 0.2 * r.normal(size=H), gpu)
    want = moe.norm(x, w, EPS, res=rs, q_mode=q)
    for swap in (False, True):
        bx, br = torch.full((T * H + 16,), 7.0, dtype=torch.bfloat16, device=gpu), torch.full((T * H + 16,), 7.0, dtype=torch.bfloat16, device=gpu)
        x2, r2 = bx[shift:shift + T * H].view(T, H), br[shift:shift + T * H].view(T, H)
        x2.copy_(x)
        r2.copy_(rs)
        got = moe.norm(x2, w, EPS, res=r2, q_mode=q, sum=r2 if swap else x2, y=x2 if swap else r2)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b)
        for buf in (bx, br):
            assert (buf[:shift] == 7).all() and (buf[shift + T * H:] == 7).all()
