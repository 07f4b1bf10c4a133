"""Calls of the FP8 products and the sampler that are refused before anything is launched (no GPU)."""
import ctypes
import os

import pytest

import moe_expert_layer_topk_amd as moe

FAKE, ODD, NULL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), None      # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from moe_expert_layer_topk_amd.build import build
        build()
    return moe.lib()


def test_products(L):
    def gemm(a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, M=4, N=8, K=256, t=0, out=FAKE):
        return L.moe_gemm_fp8(a, sa, b, sb, NULL, NULL, M, N, K, t, out, NULL)

    def glu(a=FAKE, sa=FAKE, w=FAKE, s=FAKE, M=4, I=8, K=256, h=FAKE):
        return L.moe_glu_fp8(a, sa, w, s, M, I, K, h, NULL)
    for bad in ({"a": NULL}, {"sa": NULL}, {"M": 0}, {"M": (1 << 30) + 1}, {"K": 0}, {"K": 8}, {"K": 24}, {"K": 131072}, {"a": ODD}):
        assert gemm(**bad) == -1 and glu(**bad) == -1, bad
    for bad in ({"b": NULL}, {"sb": NULL}, {"out": NULL}, {"N": 0}, {"t": 2}, {"t": -1}, {"b": ODD}, {"M": 1 << 30, "N": 256}):
        assert gemm(**bad) == -1, bad
    for bad in ({"w": NULL}, {"s": NULL}, {"h": NULL}, {"I": 0}, {"w": ODD}, {"I": 1 << 30, "M": 256}):
        assert glu(**bad) == -1, bad


def test_sample(L):
    def sample(l=FAKE, t=1, B=4, V=100, stride=100, u=FAKE, ids=FAKE):
        return L.moe_sample(l, t, B, V, stride, u, NULL, NULL, NULL, NULL, ids, FAKE, FAKE, FAKE, 1 << 40, NULL)
    for bad in ({"l": NULL}, {"u": NULL}, {"ids": NULL}, {"B": 0}, {"B": 65536}, {"V": 0, "stride": 0}, {"V": (1 << 20) + 1, "stride": 1 << 21},
                {"stride": 99}, {"stride": (1 << 40) + 1}, {"t": 2}, {"l": ctypes.c_void_p(0x1002)}, {"l": ctypes.c_void_p(0x1001), "t": 0}):
        assert sample(**bad) == -1, bad
    assert L.moe_sample_workspace_bytes(0, 100) == 0 and L.moe_sample_workspace_bytes(4, 1 << 21) == 0
    need = L.moe_sample_workspace_bytes(1, 131072)
    if need:
        short = (FAKE, 1, 1, 131072, 131072, FAKE, NULL, NULL, NULL, NULL, FAKE, FAKE, FAKE)
        assert L.moe_sample(*short, FAKE, need - 1, NULL) == -1
        assert L.moe_sample(*short, NULL, need, NULL) == -1
        assert L.moe_sample(*short, ODD, need, NULL) == -1
