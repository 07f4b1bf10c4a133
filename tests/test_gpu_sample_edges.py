"""moe_sample at the ends of its ranges: temperatures and logits near fp32's
limits, chunks without a token, as many rows and as long offsets as allowed,
workspaces of the caller's. Decisions and tolerances as in test_gpu_sample.py; rows
whose result is the same call's on other data beside them give the same bits.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import sample as oracle_sample
from test_gpu_sample import _dev, _say

pytestmark = pytest.mark.gpu


def _against_oracle(gpu, l, u, par):
    import torch
    V = l.shape[1]
    ids, p, _ = moe.sample(_dev(l, gpu), _dev(u, gpu), *(_dev(v, gpu) for v in par))
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        rid, rp, margin = oracle_sample(l.astype(np.float64), u.astype(np.float64), *(None if v is None else v.astype(np.float64) for v in par))
    sure = margin > V * 2.0 ** -42
    _say(f"    {int(sure.sum())} of {len(rid)} decided")
    assert np.array_equal(ids.cpu().numpy()[sure], rid[sure])
    assert np.all(np.abs(p.double().cpu().numpy() - rp)[sure] <= rp[sure] * (2.0 ** -24 + V * 2.0 ** -42))
    return sure


@pytest.mark.parametrize("V", [700, 9000, 131072])
@pytest.mark.parametrize("size", [1e-3, 1.0, 1e4, 8e37])
def test_temperatures(gpu, V, size):
    """From the smallest subnormal to infinity, beside logits whose differences reach fp32's largest."""
    f = np.float32
    t = np.array([1e-45, 1e-40, 1e-38, 1e-30, 1e-9, 1e-3, 1e3, 1e9, 1e30, 3.4e38, np.inf], dtype=f)
    B = len(t)
    r = np.random.default_rng([11, V])
    l = np.clip(r.normal(size=(B, V)) * size, -3.3e38, 3.3e38).astype(f)
    l[:, 5] = 0.0
    u = r.random(B).astype(f)
    decided = 0
    for k, pp, mp in ((None, None, None), (40, None, None), (None, 0.9, None), (None, None, 0.05), (3000, 0.95, 0.001), (None, 0.6, 0.3)):
        _say(f"[temperature] V={V} logits of {size} k={k} p={pp} m={mp}")
        par = [t, None if k is None else np.full(B, k, np.int32), None if pp is None else np.full(B, pp, f), None if mp is None else np.full(B, mp, f)]
        decided += _against_oracle(gpu, l, u, par).mean()
    assert decided > 0.9 * 6


@pytest.mark.parametrize("V,masked", [(40001, [(0, 12288)]), (40001, [(4096, 8192), (36864, 40001)]), (131072, [(0, 131071)]), (131072, [(1, 131072)]),
                                      (9000, [(100, 8999)])])
def test_chunks_without_a_token(gpu, V, masked):
    f = np.float32
    B = 6
    r = np.random.default_rng([12, V, len(masked)])
    l = (r.normal(size=(B, V)) * np.array([0.001, 1, 4] * 2)[:, None]).astype(f)
    for lo, hi in masked:
        l[:, lo:hi] = -np.inf
    u = r.random(B).astype(f)
    one = np.ones(B, f)
    for par in ([one, None, None, None], [one, np.full(B, 5, np.int32), None, None], [one, None, one * f(0.9), None], [one, None, one * f(0.999), one * f(1e-5)],
                [one, np.full(B, 3000, np.int32), one * f(0.9), None], [one * 0, None, None, None]):
        _say(f"[masked chunks] V={V} {masked} {[None if v is None else float(v[0]) for v in par]}")
        assert _against_oracle(gpu, l, u, par).mean() > 0.6


@pytest.mark.parametrize("V", [20000, 131072, 300007])
def test_min_p_among_many(gpu, V):
    """Rows from flat to peaked whose last kept token is top_p's or min_p's, thousands of tokens behind the first, near it, or the first."""
    f = np.float32
    B = 12
    r = np.random.default_rng([14, V])
    l = (r.normal(size=(B, V)) * np.array([0.02, 0.3, 0.8, 1.2, 2, 3] * 2)[:, None]).astype(f)
    l[6:] += f(100)
    for pp, mp in ((0.97, 1e-4), (0.99, 1e-3), (0.9, 0.01), (0.999, 0.05), (0.6, 0.3), (0.95, 0.9), (0.9, 1.0), (0.9999, 1e-9), (0.8, 1e-30)):
        _say(f"[min_p] V={V} p={pp} m={mp}")
        par = [(0.7 + 0.8 * r.random(B)).astype(f), None, np.full(B, pp, f), np.full(B, mp, f)]
        # (A demand on the rows, not on the call. Some decide nothing: 2^-45 on both sides of a min_p of 1e-9 is 5.7e-5 of
        # it, and rows of 131072 have some 2000 tokens for each factor of e there; V 2^-42 = 7e-8 on both sides of top_p's
        # border reaches the next token where the border's weights are 1e-6 and less, as in long peaked rows with 0.999.)
        assert _against_oracle(gpu, l, r.random(B).astype(f), par).mean() >= 0.5


def test_workspaces(gpu):
    """The caller's: exact, larger, with anything in it; too small or off its alignment is refused. Calls on two streams at once have one each."""
    import torch
    r = np.random.default_rng(13)
    sets = []
    for B, V in ((1, 131072), (40, 20011)):
        need = moe.sample_workspace_bytes(B, V)
        assert need > 0 and need % 8 == 0
        l = torch.from_numpy((r.normal(size=(B, V)) * 2).astype(np.float32)).to(gpu)
        u = torch.from_numpy(r.random(B).astype(np.float32)).to(gpu)
        t, pp = torch.full((B,), 1.3, device=gpu), torch.full((B,), 0.97, device=gpu)
        ids, p, _ = moe.sample(l, u, t, top_p=pp)
        for size, fill in ((need, 0), (need + 1000, 255), (need, 127)):
            ws = torch.full((size,), fill, dtype=torch.uint8, device=gpu)
            got = moe.sample(l, u, t, top_p=pp, ws=ws)
            assert torch.equal(got[0], ids) and torch.equal(got[1], p)
        big = torch.zeros(need + 512, dtype=torch.uint8, device=gpu)
        for ws in (big[:need - 1], big[8:need + 8], big[:0]):
            with pytest.raises(moe.MoeError):
                moe.sample(l, u, t, top_p=pp, ws=ws)
        sets.append((l, u, t, pp, ids, p))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(gpu) for _ in sets]
    spaces = [torch.empty(moe.sample_workspace_bytes(*s[0].shape), dtype=torch.uint8, device=gpu) for s in sets]
    torch.cuda.synchronize()
    got = [[moe.sample(l, u, t, top_p=pp, ws=ws, stream=st) for (l, u, t, pp, _, _), ws, st in zip(sets, spaces, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for one in got:
        for (ids, p, _), s in zip(one, sets):
            assert torch.equal(ids, s[4]) and torch.equal(p, s[5])


@pytest.mark.parametrize("V", [3, 5000])
def test_as_many_rows_as_allowed(gpu, V):
    import torch
    B = 65535
    _say(f"[rows] {B} x {V}")
    g = torch.Generator(device=gpu)
    g.manual_seed(1)
    l = torch.randn(B, V, device=gpu, generator=g)
    u = torch.rand(B, device=gpu, generator=g)
    pp = torch.full((B,), 0.9, device=gpu)
    ids, p, _ = moe.sample(l, u, top_p=pp)
    for part in (slice(0, 300), slice(32700, 32900), slice(B - 300, B)):
        few = moe.sample(l[part], u[part], top_p=pp[part])
        assert torch.equal(ids[part], few[0]) and torch.equal(p[part], few[1])
    more = torch.zeros(B + 1, V, device=gpu)
    with pytest.raises(moe.MoeError):
        moe.sample(more, torch.zeros(B + 1, device=gpu))
    torch.cuda.synchronize()


@pytest.mark.parametrize("B,V,stride,bf16", [(33000, 131072, 131080, True), (4200, 1000, 1 << 20, True), (1100, 9001, (1 << 22) + 1, False)])
def test_logits_past_2_to_the_32(gpu, B, V, stride, bf16):
    """4.3e9 elements and more between the first row and the last."""
    import torch
    assert (B - 1) * stride > 2 ** 32
    _say(f"[large logits] {B} x {V}, rows {stride} apart")
    dt = torch.bfloat16 if bf16 else torch.float32
    l = torch.empty((B - 1) * stride + V, dtype=dt, device=gpu).as_strided((B, V), (stride, 1))
    g = torch.Generator(device=gpu)
    g.manual_seed(2)
    for r in range(0, B, 2000):
        l[r:r + 2000] = torch.randn(min(2000, B - r), V, device=gpu, generator=g).to(dt)
    u = torch.rand(B, device=gpu, generator=g)
    t, pp = torch.full((B,), 0.6, device=gpu), torch.full((B,), 0.8, device=gpu)
    for par in ([t], [t, None, pp]):
        ids, p, _ = moe.sample(l, u, *par)
        torch.cuda.synchronize()
        assert bool(((ids >= 0) & (ids < V)).all())
        pick = torch.tensor(sorted({0, 1, B // 2, B - 2, B - 1} | {min(b // stride + d, B - 1) for b in (2 ** 30, 2 ** 31, 2 ** 32) for d in (0, 1)}), device=gpu)
        few = moe.sample(l[pick], u[pick], *(None if v is None else v[pick] for v in par))
        assert torch.equal(ids[pick], few[0]) and torch.equal(p[pick], few[1])
