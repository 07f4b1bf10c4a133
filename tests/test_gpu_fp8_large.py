"""FP8 products whose byte and element offsets pass 2^31 and 2^32.

Codes of whole numbers up to 2 and scales of 1 and 2: products and their sums are
whole numbers below 2^24, exact in fp32 however they are grouped. Rows at the start, at
the end and on both sides of the offsets are checked against fp64.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from test_gpu_dense import _say
from test_gpu_dense_large import _rows_around

pytestmark = pytest.mark.gpu

CODES = [0x00, 0x38, 0xB8, 0x40, 0xC0]                                # 0, 1, -1, 2, -2


def _codes(gpu, rows, cols, seed):
    """Random codes, made on the device in pieces."""
    import torch
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    table = torch.tensor(CODES, dtype=torch.uint8, device=gpu)
    t = torch.empty(rows, cols, dtype=torch.uint8, device=gpu)
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        t[r:r + step] = table[torch.randint(0, 5, (min(step, rows - r), cols), device=gpu, generator=g)]
    return t


def _values(codes):
    v = np.zeros(256)
    v[CODES] = [0, 1, -1, 2, -2]
    return v[codes.cpu().numpy()]


def _scales(gpu, rows, K, seed):
    """E8M0 bytes of 1 and 2, [rows, blocks]."""
    import torch
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    return torch.randint(127, 129, (rows, (K + 127) // 128), dtype=torch.uint8, device=gpu, generator=g)


def _scaled(values, powers, K):
    return values * np.repeat(powers, 128, axis=1)[:, :K]


@pytest.mark.parametrize("few", [24, 300])
@pytest.mark.parametrize("tall", ["a", "b"])
@pytest.mark.parametrize("f32", [True, False])
def test_operand_past_4_gib(gpu, tall, few, f32):
    """a or b of 5.2 GB; |sums| <= 131056 * 4 * 4 < 2^21."""
    import torch
    n, K = 40009, 131056
    assert n * K > 2 ** 32
    _say(f"[large FP8 product] {tall} {n} x {K}, other {few}, fp32 {f32}")
    M, N = (n, few) if tall == "a" else (few, n)
    a, b = _codes(gpu, M, K, 1), _codes(gpu, N, K, 2)
    sa = _scales(gpu, M, K, 3)
    sb = (_scales(gpu, (N + 127) // 128, K, 4) - 126).float()
    out = moe.gemm_fp8(a, sa, b, sb, out_dtype=torch.float32 if f32 else torch.bfloat16)
    torch.cuda.synchronize()
    pick = _rows_around(n, K, 2 ** 31, 2 ** 32)
    rows, cols = (pick, list(range(N))) if tall == "a" else (list(range(M)), pick)
    x = _scaled(_values(a[rows]), sa[rows].cpu().numpy() - 126.0, K)
    y = _scaled(_values(b[cols]), sb[[c // 128 for c in cols]].cpu().numpy().astype(np.float64), K)
    want = torch.from_numpy(x @ y.T).float()
    got = out[rows][:, cols].cpu()
    assert torch.equal(got, want if f32 else want.to(torch.bfloat16))


def test_gated_operand_past_4_gib(gpu):
    """w13 of 5.2 GB, whose up rows lie past 2^31 bytes: equal rows give equal outputs to a small call's."""
    import torch
    I, K, M = 20005, 131056, 40
    assert 2 * I * K > 2 ** 32
    _say(f"[large gated FP8 product] w13 {2 * I} x {K}")
    w, a = _codes(gpu, 2 * I, K, 5), _codes(gpu, M, K, 6)
    sa = _scales(gpu, M, K, 7)
    KB, IB = (K + 127) // 128, (I + 127) // 128
    h = moe.glu_fp8(a, sa, w, torch.full((2 * IB, KB), 2.0 ** -12, device=gpu))
    pick = _rows_around(I, K, 2 ** 31, 2 ** 32 - I * K)
    rows = torch.tensor(pick + [I + i for i in pick], device=gpu)
    want = moe.glu_fp8(a, sa, w[rows], torch.full((2, KB), 2.0 ** -12, device=gpu))
    torch.cuda.synchronize()
    assert torch.equal(h[:, pick], want)


@pytest.mark.parametrize("N", [16392, 16389])
def test_output_past_4_gib(gpu, N):
    """2^31 outputs, 4.3 GB (aligned rows and not), added in place."""
    import torch
    M, K = 131101, 16
    assert M * N > 2 ** 31
    _say(f"[large FP8 output] {M} x {N}")
    a, b = _codes(gpu, M, K, 8), _codes(gpu, N, K, 9)
    sa = _scales(gpu, M, K, 10)
    sb = (_scales(gpu, (N + 127) // 128, K, 11) - 126).float()
    out = torch.full((M, N), 2.0, dtype=torch.bfloat16, device=gpu)
    moe.gemm_fp8(a, sa, b, sb, add=out, out=out)
    torch.cuda.synchronize()
    pick = _rows_around(M, N, 2 ** 30, 2 ** 31)
    x = _scaled(_values(a[pick]), sa[pick].cpu().numpy() - 126.0, K)
    y = _values(b) * np.repeat(sb.cpu().numpy().astype(np.float64), 128, axis=0)[:N]
    assert torch.equal(out[pick].cpu(), torch.from_numpy(x @ y.T + 2).float().to(torch.bfloat16))


@pytest.mark.parametrize("M,N", [((1 << 26) + 1, 1), (1, (1 << 26) + 3)])
def test_one_side_very_long(gpu, M, N):
    """Outputs narrower than a lane's columns, and a million tiles in a row."""
    import torch
    K = 16
    _say(f"[long FP8 product] {M} x {N}")
    a, b = _codes(gpu, M, K, 12), _codes(gpu, N, K, 13)
    sa, sb = _scales(gpu, M, K, 14), (_scales(gpu, (N + 127) // 128, K, 15) - 126).float()
    out = moe.gemm_fp8(a, sa, b, sb)
    table = torch.zeros(256, device=gpu)
    table[CODES] = torch.tensor([0.0, 1.0, -1.0, 2.0, -2.0], device=gpu)
    if N == 1:
        want = (table[a.long()] * table[b.long()]).sum(1, keepdim=True) * (sa.float() - 126) * sb
    else:
        want = ((table[b.long()] * table[a.long()]).sum(1) * sb[torch.arange(N, device=gpu) // 128, 0] * (sa.float() - 126)[0])[None]
    torch.cuda.synchronize()
    assert torch.equal(out, want.to(torch.bfloat16))
