"""moe_sample against the fp64 oracle.

Each weight is off by half of 2^-42 of the largest, and fp64's exponential by
far less, so no sum of V weights is off by more than V 2^-43, and a decision
(a border, the draw) by twice that: where the oracle's decisions are more than
V 2^-42 away from going the other way, the ids are equal. (w >= min_p is one
weight's decision: the exponential is off by less than 1e-14 = 2^-46.5 of it, so
2^-45 is enough there.) p is a quotient of
fp64 values, off by the sums' V 2^-43 (of a sum of at least 1) and one rounding
to fp32: p (2^-24 + V 2^-42).
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from oracle import sample as oracle_sample
from oracle.sample import sample_row

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


def _dev(a, dev, dtype=None):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev).to(dtype or (torch.float32 if a.dtype.kind == "f" else torch.int32))


def _check(ids, p, ref, V, kept_of=None):
    rid, rp, margin = ref
    sure = margin > V * 2.0 ** -42
    ids, p = ids.cpu().numpy(), p.double().cpu().numpy()
    _say(f"    {int(sure.sum())} of {len(rid)} rows decided, smallest margin {margin.min():.2e}")
    assert sure.mean() > 0.9
    assert np.array_equal(ids[sure], rid[sure])
    assert np.all(np.abs(p - rp)[sure] <= rp[sure] * (2.0 ** -24 + V * 2.0 ** -42))


def _parameters(r, B, t, k, p, m):
    f = np.float32
    temp = np.where(r.random(B) < 0.15, 0, 0.3 + 1.2 * r.random(B)).astype(f) if t else None
    top_k = np.where(r.random(B) < 0.2, 0, np.exp(7 * r.random(B))).astype(np.int32) if k else None
    top_p = np.where(r.random(B) < 0.2, 1, r.random(B)).astype(f) if p else None
    min_p = (0.2 * r.random(B)).astype(f) if m else None
    return temp, top_k, top_p, min_p


SHAPES = [(1, 1), (3, 2), (5, 63), (4, 64), (7, 65), (2, 1023), (9, 1024), (3, 1025), (2, 4097), (33, 5000), (5, 32768), (1, 50021), (16, 50021),
          (1, 131072), (4, 200003), (300, 700), (2, 1 << 20)]


@pytest.mark.parametrize("B,V", SHAPES)
@pytest.mark.parametrize("which", [(0, 0, 0, 0), (1, 0, 0, 0), (1, 1, 0, 0), (1, 0, 1, 0), (0, 0, 0, 1), (1, 1, 1, 1)])
@pytest.mark.parametrize("bf16", [False, True])
def test_sample(gpu, B, V, which, bf16):
    import torch
    r = np.random.default_rng([1, B, V, *which])
    _say(f"[sample] B={B} V={V} t,k,p,m={which} bf16={bf16}")
    l = torch.from_numpy((r.normal(size=(B, V)) * 2.5).astype(np.float32)).to(torch.bfloat16 if bf16 else torch.float32)
    u = r.random(B).astype(np.float32)
    par = _parameters(r, B, *which)
    ids, p, err = moe.sample(l.to(gpu), _dev(u, gpu), *(_dev(v, gpu) for v in par))
    torch.cuda.synchronize()
    assert err is None and ids.dtype == torch.int32 and p.dtype == torch.float32
    _check(ids, p, oracle_sample(l.double().numpy(), u.astype(np.float64), *(None if v is None else v.astype(np.float64) for v in par)), V)


@pytest.mark.parametrize("name", ["flat", "two values", "peaked", "wide", "steps", "tiny", "masked"])
@pytest.mark.parametrize("B,V", [(6, 1000), (3, 40001), (1, 131072)])
def test_kinds_of_rows(gpu, name, B, V):
    """Rows of one value, of ties, with one token far above, of a very wide range, with most tokens masked."""
    import torch
    r = np.random.default_rng([2, V])
    l = {"flat": np.zeros((B, V)), "two values": r.integers(0, 2, size=(B, V)) * 3.0, "peaked": r.normal(size=(B, V)), "wide": r.normal(size=(B, V)) * 1e30,
         "steps": np.floor(r.normal(size=(B, V)) * 8) / 4, "tiny": r.normal(size=(B, V)) * 1e-40,
         "masked": np.where(r.random((B, V)) < 0.99, -np.inf, r.normal(size=(B, V)))}[name]
    if name == "peaked":
        l[:, V // 3] = 60.0
    if name == "masked":
        l[:, V // 2] = 0.0
    l = l.astype(np.float32)
    for which in ((0, 0, 0, 0), (1, 1, 1, 1), (1, 0, 1, 0)):
        u = r.random(B).astype(np.float32)
        par = _parameters(r, B, *which)
        _say(f"[rows] {name} B={B} V={V} {which}")
        ids, p, _ = moe.sample(_dev(l, gpu), _dev(u, gpu), *(_dev(v, gpu) for v in par))
        torch.cuda.synchronize()
        rid, rp, margin = oracle_sample(l.astype(np.float64), u.astype(np.float64), *(None if v is None else v.astype(np.float64) for v in par))
        sure = margin > V * 2.0 ** -42
        assert np.array_equal(ids.cpu().numpy()[sure], rid[sure]), (ids, rid, margin)
        assert np.all(np.abs(p.double().cpu().numpy() - rp)[sure] <= rp[sure] * (2.0 ** -24 + V * 2.0 ** -42))
        assert sure.any() or name == "two values"


@pytest.mark.parametrize("V", [9000, 131072])
@pytest.mark.parametrize("bf16", [False, True])
def test_many_kept_tokens(gpu, V, bf16):
    """top_k of thousands, top_p of flat rows, ordered logits (one chunk has all of the firsts), soft masks: borders among more
    tokens than are kept as candidates."""
    import torch
    r = np.random.default_rng([7, V])
    B = 12
    l = r.normal(size=(B, V)) * np.array([0.01, 0.3, 1, 3] * 3)[:, None]
    l[4:8] = -np.sort(-l[4:8], axis=1)
    l[8:] = np.where(r.random((4, V)) < 0.9, np.array([-1e4, -65504.0, -3e38, -30.0])[:, None], l[8:])
    l = torch.from_numpy(l.astype(np.float32)).to(torch.bfloat16 if bf16 else torch.float32)
    for k, pp, mp in ((2000, None, None), (5000, 0.9, None), (0, 0.9, None), (0, 0.97, 1e-6), (0, 0.8, 0.02), (0, 0.9999, None), (V - 7, 0.5, 0.001), (0, 0.99, None), (0, 0.3, None), (300, None, None), (0, None, 1e-4),
                      (V + 5, None, None), (700, 0.999, None)):
        u = r.random(B).astype(np.float32)
        t = (0.2 + 2 * r.random(B)).astype(np.float32)
        par = [t, np.full(B, k, np.int32), None if pp is None else np.full(B, pp, np.float32), None if mp is None else np.full(B, mp, np.float32)]
        _say(f"[many] V={V} bf16={bf16} k={k} p={pp} m={mp}")
        ids, p, _ = moe.sample(l.to(gpu), _dev(u, gpu), *(_dev(v, gpu) for v in par))
        torch.cuda.synchronize()
        _check(ids, p, oracle_sample(l.double().numpy(), u.astype(np.float64), *(None if v is None else v.astype(np.float64) for v in par)), V)


def test_equal_logits_take_the_lowest_ids(gpu):
    """Whole numbers throughout: V equal tokens, top_k and top_p of them; u walks over all of the kept ones."""
    import torch
    for V in (8, 1000, 5000, 70000):
        l = torch.full((65, V), -1.25, device=gpu)
        u = torch.arange(65, device=gpu, dtype=torch.float32) / 64
        k = torch.full((65,), 4, dtype=torch.int32, device=gpu)
        half = torch.full((65,), 0.5, device=gpu)
        want = torch.clamp((u * 4).int(), max=3)
        ids, p, _ = moe.sample(l, u, top_k=k)
        assert torch.equal(ids, want) and torch.equal(p, torch.full_like(p, 0.25))
        ids, p, _ = moe.sample(l, u, top_k=k * 2, top_p=half, min_p=torch.ones_like(u))
        assert torch.equal(ids, want) and torch.equal(p, torch.full_like(p, 0.25))
        l[:, : V // 2] = -2.5                                     # the upper half's lowest ids
        ids, _, _ = moe.sample(l, u, top_k=k)
        assert torch.equal(ids, want + V // 2)
        l[:, 1] = -0.0
        l[:, V - 1] = 0.0                                         # equal to -0
        ids, _, _ = moe.sample(l, u, top_k=k // 4)
        assert torch.equal(ids, torch.ones_like(ids))


def test_greedy_and_the_ends_of_u(gpu):
    import torch
    r = np.random.default_rng(3)
    for dt in (torch.float32, torch.bfloat16):
        l = torch.from_numpy(r.normal(size=(40, 3001)).astype(np.float32)).to(dt).to(gpu)
        u = torch.from_numpy(r.random(40).astype(np.float32)).to(gpu)
        zero = torch.zeros(40, device=gpu)
        ids, p, _ = moe.sample(l, u, temperature=zero, top_p=u, min_p=u)
        top = l.float().max(dim=1).values[:, None]
        first = torch.where(l.float() == top, torch.arange(3001, device=gpu), 3001).min(dim=1).values
        assert torch.equal(ids.long(), first) and torch.equal(p, torch.ones_like(p))
        kept = l.float() >= torch.sort(l.float(), dim=1, descending=True).values[:, 5:6]     # six or more: ties at the border
        k = kept.sum(dim=1).to(torch.int32)
        ids, _, _ = moe.sample(l, zero, top_k=k)
        assert torch.equal(ids.long(), kept.int().argmax(dim=1))
        ids, _, _ = moe.sample(l, zero + 1, top_k=k)
        assert torch.equal(ids.long(), 3000 - kept.flip(1).int().argmax(dim=1))


def test_rows_without_a_token_and_invalid_values(gpu):
    import torch
    inf, nan = float("inf"), float("nan")
    for V in (7, 3000, 60000):
        for dt in (torch.float32, torch.bfloat16):
            B = 14
            l = torch.zeros(B, V, dtype=dt, device=gpu)
            l[:, V - 1] = 5
            u, t, pp, mp = (torch.full((B,), v, device=gpu) for v in (0.5, 1.0, 0.9, 0.01))
            k = torch.full((B,), 3, dtype=torch.int32, device=gpu)
            l[1], l[2, V // 2], l[3, 0], l[4, V - 1] = -inf, nan, inf, -nan
            l[5, : V - 1] = -inf                                  # one token left
            u[6], u[7], u[8] = nan, -0.1, 1.5
            t[9], t[10] = -1.0, nan
            pp[11], mp[12], mp[13] = nan, nan, 1.01
            err = torch.full((1,), 100, dtype=torch.int32, device=gpu)
            ids, p, e = moe.sample(l, u, t, k, pp, mp, err=err)
            torch.cuda.synchronize()
            good = [0, 5]
            assert e is err and int(err) == 100 + B - 2
            for r in range(B):
                want = V - 1 if r in good else -1
                assert int(ids[r]) == want, (V, dt, r)
                assert (float(p[r]) > 0) == (r in good)
    # parameters that are allowed: infinite temperature, negative top_k, min_p and top_p, top_p above 1
    l = torch.arange(8, device=gpu, dtype=torch.float32)[None].repeat(5, 1) * 3
    l[:, 0] = -inf
    one = torch.ones(5, device=gpu)
    t = torch.tensor([inf, 1, 1, 1, 1], device=gpu)
    k = torch.tensor([0, -5, 0, 0, 100], dtype=torch.int32, device=gpu)
    pp = torch.tensor([1, 1, -1.0, 2, 1], device=gpu)
    mp = torch.tensor([0, 0, 0, -3.0, 0], device=gpu)
    ids, p, _ = moe.sample(l, one * 0.0, t, k, pp, mp)
    assert ids.tolist() == [1, 1, 7, 1, 1] and abs(float(p[0]) - 1 / 7) < 1e-7 and float(p[2]) == 1


def test_strides_outputs_and_streams(gpu):
    """Rows inside longer ones, at any element; outputs passed; another stream; two calls at once."""
    import torch
    r = np.random.default_rng(4)
    for dt in (torch.float32, torch.bfloat16):
        for B, V, width, off in ((5, 1001, 1100, 0), (5, 1001, 1003, 1), (3, 50021, 50176, 3), (1, 777, 1000, 5), (40, 130, 131, 1)):
            wide = torch.from_numpy((r.normal(size=(B, width)) * 3).astype(np.float32)).to(dt).to(gpu)
            l = wide[:, off:off + V]
            if off:
                wide[:, :off] = float("nan")
            wide[:, off + V:] = float("inf")
            u = torch.from_numpy(r.random(B).astype(np.float32)).to(gpu)
            t = torch.full((B,), 0.8, device=gpu)
            want = moe.sample(l.contiguous(), u, t)
            ids, p = torch.full((B,), 9, dtype=torch.int32, device=gpu), torch.zeros(B, device=gpu)
            got = moe.sample(l, u, t, ids=ids, p=p)
            assert got[0] is ids and got[1] is p
            side = torch.cuda.Stream(gpu)
            side.wait_stream(torch.cuda.current_stream(gpu))
            there = moe.sample(l, u, t, stream=side)
            again = moe.sample(l, u, t)
            torch.cuda.synchronize()
            for x in (got, there, again):
                assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
            assert bool((want[0] >= 0).all())


def test_captured_and_replayed(gpu):
    """A graph with several calls, its inputs changed between replays, each replay against an eager call."""
    import torch
    r = np.random.default_rng(5)
    sets = []
    for B, V in ((1, 131072), (3, 50021), (20, 4000), (300, 1000)):
        l = torch.empty(B, V, device=gpu)
        sets.append((l, torch.empty(B, device=gpu), torch.full((B,), 0.9, device=gpu), torch.full((B,), 50, dtype=torch.int32, device=gpu),
                     torch.full((B,), 0.95, device=gpu), torch.full((B,), 0.02, device=gpu),
                     torch.empty(B, dtype=torch.int32, device=gpu), torch.empty(B, device=gpu)))

    def fill():
        for l, u, *_ in sets:
            l.copy_(torch.from_numpy((r.normal(size=tuple(l.shape)) * 3).astype(np.float32)))
            u.copy_(torch.from_numpy(r.random(u.numel()).astype(np.float32)))
    fill()
    for s in sets:
        moe.sample(*s[:6])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for l, u, t, k, pp, mp, ids, p in sets:
            moe.sample(l, u, t, k, pp, mp, ids=ids, p=p)
            moe.sample(l, u, t, ids=ids, p=p)
            moe.sample(l, u, t, k, pp, mp, ids=ids, p=p)
    for _ in range(5):
        fill()
        want = [moe.sample(*s[:6])[:2] for s in sets]
        g.replay()
        torch.cuda.synchronize()
        for (wi, wp), (*_, ids, p) in zip(want, sets):
            assert torch.equal(wi, ids) and torch.equal(wp, p)


def test_next_token(gpu):
    """A decode step's end: norm to e4m3 rows, the head's logits, a token; against the same logits through the oracle."""
    import torch
    r = np.random.default_rng(6)
    for T, H, V in ((1, 256, 1000), (9, 512, 5003), (70, 256, 2048)):
        x = torch.from_numpy(r.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).to(gpu)
        _, _, a, sa = moe.norm(x, None, 1e-6, q_mode=moe.Q_FP8_G128_POW2, with_y=False)
        w = torch.from_numpy((r.integers(0, 0x70, size=(V, H)) + 128 * r.integers(0, 2, size=(V, H))).astype(np.uint8)).to(gpu)
        s = torch.full(((V + 127) // 128, H // 128), 0.002, device=gpu)
        u = torch.from_numpy(r.random(T).astype(np.float32)).to(gpu)
        t, pp = torch.full((T,), 0.7, device=gpu), torch.full((T,), 0.9, device=gpu)
        ids, p, logits = moe.next_token(a, sa, w, s, u, temperature=t, top_p=pp)
        side = torch.cuda.Stream(gpu)
        side.wait_stream(torch.cuda.current_stream(gpu))
        there = moe.next_token(a, sa, w, s, u, temperature=t, top_p=pp, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(logits, moe.gemm_fp8(a, sa, w, s, out_dtype=torch.float32))
        assert torch.equal(there[0], ids) and torch.equal(there[2], logits)
        _check(ids, p, oracle_sample(logits.double().cpu().numpy(), u.double().cpu().numpy(), t.double().cpu().numpy(), None,
                                     pp.double().cpu().numpy()), V)


def test_refusals(gpu):
    import torch
    l, u = torch.zeros(4, 100, device=gpu), torch.zeros(4, device=gpu)
    moe.sample(l, u)
    for bad in (l.cpu(), l.double(), l.half(), l.t(), l[:, ::2], l[0], l[:0], torch.zeros(100, device=gpu).expand(4, 100), None,
                torch.zeros(4, (1 << 20) + 1, device=gpu)):
        with pytest.raises(moe.MoeError):
            moe.sample(bad, u)
    for kw in ({"u": u[:3]}, {"u": u.cpu()}, {"u": None}, {"u": u.double()}, {"temperature": u.half()}, {"top_k": u}, {"top_k": torch.zeros(4, dtype=torch.int64, device=gpu)},
               {"top_p": u[:, None]}, {"min_p": torch.zeros(8, device=gpu)[::2]}, {"ids": torch.zeros(4, device=gpu)}, {"p": torch.zeros(3, device=gpu)},
               {"err": torch.zeros(1, device=gpu)}, {"err": torch.zeros(2, dtype=torch.int32, device=gpu)}, {"ws": torch.zeros(4, device=gpu)}):
        with pytest.raises(moe.MoeError):
            moe.sample(l, **{"u": u, **kw})
    assert sample_row(np.zeros(3), 0.5)[0] == 1
