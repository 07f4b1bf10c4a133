"""Pins of the dense-operator oracle (hand values, invariants, special cases)
and the host checks of their C-ABI calls (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import dense


def test_rms_norm_by_hand():
    # v = (3, -4, 0, 0) + (0, 0, 12, 0): mean square 169 / 4, r = 2 / 13
    y, v = dense.rms_norm([[3, -4, 0, 0]], [1, 2, 0.5, 7], 0.0, res=[[0, 0, 12, 0]])
    assert np.array_equal(v, [[3, -4, 12, 0]])
    assert np.allclose(y, [[6 / 13, -16 / 13, 12 / 13, 0]], rtol=1e-15, atol=0)
    # eps enters under the root: mean square 3, eps 1 -> r = 1/2
    y, _ = dense.rms_norm([[3, 0, 0]], None, 1.0)
    assert np.allclose(y, [[1.5, 0, 0]], rtol=1e-15, atol=0)


def test_rms_norm_has_unit_mean_square():
    x = np.random.default_rng(0).normal(size=(5, 37)) * 10
    y, _ = dense.rms_norm(x, None, 0.0)
    assert np.allclose(np.mean(y * y, axis=1), 1.0, rtol=1e-13)


def test_i8_rows_by_hand():
    t, s = dense.i8_rows(np.array([[127.0, -1.5, 0.25], [0.0, 0.0, 0.0], [-254.0, 2.0, 1.0]]))
    assert np.array_equal(np.rint(t[0]), [127, -2, 0]) and s[0] == 1.0
    assert np.array_equal(t[1], [0, 0, 0]) and 0 < s[1] <= 2.0 ** -100
    assert np.array_equal(np.rint(t[2]), [-127, 1, 0]) and s[2] == 2.0


def test_gemm_by_hand_and_against_integers():
    p, o = dense.gemm_i8(np.array([[1, 2], [-128, 3]], np.int8), [0.5, 2], np.array([[4, 5], [-6, 127], [0, 1]], np.int8),
                         [1, 0.25, 3], bias=[1, 0, 0], add=[[0, 0, 1], [0, 0, 0]])
    # sums: (14, 248, 2), (-497, 1149, 3)
    assert np.array_equal(p, [[7, 31, 3], [-994, 574.5, 18]])
    assert np.array_equal(o, [[8, 31, 4], [-993, 574.5, 18]])
    r = np.random.default_rng(1)
    a, b = r.integers(-128, 128, (9, 640), dtype=np.int8), r.integers(-128, 128, (7, 640), dtype=np.int8)
    p, _ = dense.gemm_i8(a, np.ones(9), b, np.ones(7))
    assert np.array_equal(p.astype(np.int64), a.astype(np.int64) @ b.astype(np.int64).T)


def test_glu_by_hand():
    # g = 0 gives 0; a large gate passes u * g; a very negative one gives 0
    w = np.array([[0, 0], [1, 0], [-1, 0], [1, 1], [1, 1], [1, 1]], np.int8)
    g, u, h = dense.glu_i8(np.array([[100, 3]], np.int8), [1.0], w, np.ones(6))
    assert np.array_equal(g, [[0, 100, -100]]) and np.array_equal(u, [[103, 103, 103]])
    assert h[0, 0] == 0 and abs(h[0, 1] - 10300) < 1e-9 and abs(h[0, 2]) < 1e-38


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from moe_expert_layer_topk_amd.build import build
        build()
    return moe.lib()


def test_missing_marshal_module_fails_loudly(L, monkeypatch):
    import sys
    from moe_expert_layer_topk_amd import binding
    monkeypatch.setattr(binding, "_marshal", None)
    monkeypatch.setitem(sys.modules, "moe_expert_layer_topk_amd._marshal", None)
    monkeypatch.delattr(moe, "_marshal", raising=False)
    with pytest.raises(moe.MoeError, match="_marshal"):
        moe.quant_rows(None)


def test_norm_host_checks(L):
    f, n, odd = ctypes.c_void_p(0x1000), None, ctypes.c_void_p(0x1002)     # never dereferenced
    ok = dict(x=f, res=n, w=n, eps=1e-6, rows=4, cols=256, q=0, sum=n, y=f, codes=n, scales=n)

    def call(**k):
        a = {**ok, **k}
        return L.moe_norm(a["x"], a["res"], a["w"], a["eps"], a["rows"], a["cols"], a["q"], a["sum"], a["y"], a["codes"],
                          a["scales"], n)

    for bad in (dict(x=n), dict(rows=0), dict(rows=-1), dict(cols=0), dict(cols=16385), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(q=3), dict(q=-1),
                dict(y=n), dict(codes=f), dict(scales=f),                     # nothing to write; codes without a mode
                dict(sum=f), dict(q=1), dict(q=1, codes=f), dict(q=1, scales=f),   # sum is y; missing codes or scales
                dict(q=2, codes=f, scales=f, cols=200), dict(q=2, codes=f, scales=f, x=odd),
                dict(q=2, codes=f, scales=f, w=odd)):
        assert call(**bad) == -1, bad
    q = ctypes.c_void_p(0x2000)
    for bad in ((n, 4, 64, f, q), (f, 0, 64, f, q), (f, 4, 0, f, q), (f, 4, 16385, f, q), (f, 4, 64, n, q), (f, 4, 64, f, n)):
        assert L.moe_quant_rows(*bad, n) == -1, bad


def test_dequant_rows_host_checks(L):
    f, n, odd = ctypes.c_void_p(0x1000), None, ctypes.c_void_p(0x1008)
    for bad in ((n, f, 4, 64, 1, f), (f, n, 4, 64, 1, f), (f, f, 4, 64, 1, n), (f, f, 0, 64, 1, f), (f, f, 4, 0, 1, f),
                (f, f, 4, 16385, 1, f), (f, f, 4, 64, 0, f), (f, f, 4, 64, 3, f), (f, f, 4, 64, 2, f), (odd, f, 4, 128, 2, f),
                (f, f, 4, 128, 2, odd), (f, f, 1 << 21, 16384, 1, f), (odd, f, 1 << 18, 16384, 1, f)):
        assert L.moe_dequant_rows(*bad, n) == -1, bad


def test_product_host_checks(L):
    f, n, odd = ctypes.c_void_p(0x1000), None, ctypes.c_void_p(0x1008)
    ok = dict(a=f, sa=f, b=f, sb=f, M=4, N=32, K=64, t=0, out=f)

    def gemm(**k):
        v = {**ok, **k}
        return L.moe_gemm_i8(v["a"], v["sa"], v["b"], v["sb"], n, n, v["M"], v["N"], v["K"], v["t"], v["out"], n)

    def glu(**k):
        v = {**ok, **k}
        return L.moe_glu_i8(v["a"], v["sa"], v["b"], v["sb"], v["M"], v["N"], v["K"], v["out"], n)

    for bad in (dict(a=n), dict(sa=n), dict(b=n), dict(sb=n), dict(out=n), dict(a=odd), dict(b=odd), dict(M=0), dict(N=0),
                dict(K=0), dict(K=8), dict(K=72), dict(K=131072), dict(M=1 << 30, N=1 << 30), dict(M=(1 << 30) + 1, N=1)):
        assert gemm(**bad) == -1, bad
        assert glu(**bad) == -1, bad
    assert gemm(t=2) == -1 and gemm(t=-1) == -1


def test_binding_refuses_before_a_launch():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    a = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.zeros(4)
    for call in (lambda: moe.norm(None), lambda: moe.norm(3), lambda: moe.gemm_i8(a, s, None, s), lambda: moe.gemm_i8(a, None, a, s),
                 lambda: moe.norm(x), lambda: moe.quant_rows(x), lambda: moe.dequant_rows(a, s), lambda: moe.dequant_rows(None, s), lambda: moe.gemm_i8(a, s, a, s),
                 lambda: moe.glu_i8(a, s, a, s), lambda: moe.norm(x[0]), lambda: moe.quant_rows(x[:0]),
                 lambda: moe.glu_i8(a, s, a[:3], s[:3])):
        with pytest.raises(moe.MoeError):
            call()


def test_launches_past_their_thread_count_are_refused(L):
    """Sizes whose grid would hold 2^32 threads: a workgroup of 256 per row, or one thread per 8 codes (unaligned: per code)."""
    f, g, n, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x2000), None, ctypes.c_void_p(0x1008)
    for rows in (1 << 24, (1 << 31) - 1):
        assert L.moe_norm(f, n, n, 1e-6, rows, 8, 0, n, g, n, n, n) == -1
        assert L.moe_quant_rows(f, rows, 8, g, g, n) == -1
    for codes, rows, cols in ((f, 1 << 20, 16384), (odd, 1 << 20, 2048), (f, 1 << 22, 516)):
        assert L.moe_dequant_rows(codes, f, rows, cols, 1, g, n) == -1
