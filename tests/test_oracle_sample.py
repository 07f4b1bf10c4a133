"""The sampling oracle and the FP8 products' oracle by hand and against sums written out."""
import numpy as np
import pytest

from oracle import dense, sample
from oracle.sample import sample_row

L2, L3 = np.log(2.0), np.log(3.0)


def test_filters_by_hand():
    # weights 1, 1/2, 1/4, 1/4, 1/8 at ids 2, 0, 1, 4, 3
    l = np.log([0.5, 0.25, 1.0, 0.125, 0.25])
    assert sample_row(l, 0.0)[2].tolist() == [2, 0, 1, 4, 3]
    assert sample_row(l, 0.0, top_k=3)[2].tolist() == [2, 0, 1]            # of the equal ids 1 and 4 the lower
    assert sample_row(l, 0.0, min_p=0.26)[2].tolist() == [2, 0]
    # all weigh 17/8: before the third token lie 12/17 = 0.7058..
    assert sample_row(l, 0.0, top_p=0.70)[2].tolist() == [2, 0]
    assert sample_row(l, 0.0, top_p=0.71)[2].tolist() == [2, 0, 1]
    # of the first three (7/4) the first is 4/7 = 0.571..
    assert sample_row(l, 0.0, top_k=3, top_p=0.57)[2].tolist() == [2]
    assert sample_row(l, 0.0, top_k=3, top_p=0.58)[2].tolist() == [2, 0]
    assert sample_row(l, 0.0, top_p=0.0)[2].tolist() == [2]


@pytest.mark.parametrize("u,want", [(0.0, 0), (0.23, 0), (0.24, 1), (0.34, 1), (0.36, 2), (0.82, 2), (0.83, 3), (0.87, 3), (0.89, 4), (1.0, 4)])
def test_draw_by_hand(u, want):
    # by id 4, 2, 8, 1, 2 seventeenths: ends at 0.235, 0.353, 0.824, 0.882, 1
    l = np.log([0.5, 0.25, 1.0, 0.125, 0.25])
    i, p, _, _ = sample_row(l, u)
    assert i == want and abs(p - [4, 2, 8, 1, 2][i] / 17) < 1e-15


def test_temperature_masks_and_rows_without_a_token():
    inf, nan = np.inf, np.nan
    assert sample_row([L2, 0.0], 0.79, temperature=0.5)[0] == 0 and sample_row([L2, 0.0], 0.81, temperature=0.5)[0] == 1   # 4 : 1
    assert sample_row([0.0, 5.0, 5.0], 0.9, temperature=0.0)[:2] == (1, 1.0)
    assert sample_row([-inf, 1.0, -inf], 0.99)[:2] == (1, 1.0)
    for l, kw in (([-inf, -inf], {}), ([0.0, nan], {}), ([0.0, inf], {}), ([0.0], {"temperature": -1.0}), ([0.0], {"top_p": nan}),
                  ([0.0], {"min_p": 1.5}), ([0.0], {"min_p": nan}), ([0.0], {"temperature": nan})):
        assert sample_row(l, 0.5, **kw)[0] == -1
    for u in (-0.1, 1.1, nan):
        assert sample_row([0.0], u)[0] == -1


def test_rows_take_their_own_parameters():
    l = np.log([[1.0, 2.0, 1.0]] * 4)
    ids, p, _ = sample(l, [0.99, 0.99, 0.99, 0.1], temperature=[1, 0, 1, 1], top_k=[0, 0, 2, 0], top_p=[1, 1, 1, 0.4], min_p=[0, 0, 0, 0])
    assert ids.tolist() == [2, 1, 1, 1] and np.allclose(p, [0.25, 1, 2 / 3, 1])


def test_draws_follow_the_weights():
    """Equidistant u give each token its share, to one part."""
    r = np.random.default_rng(3)
    l = r.normal(size=40) * 2
    n = 4000
    ids, p, _ = sample(np.repeat(l[None], n, 0), (np.arange(n) + 0.5) / n, top_k=np.full(n, 25))
    w = np.exp(l)
    w[np.argsort(-l)[25:]] = 0
    share = np.bincount(ids, minlength=40) / n
    assert np.abs(share - w / w.sum()).max() <= 1.0 / n


def test_fp8_product_by_sums():
    r = np.random.default_rng(4)
    M, N, K = 3, 130, 144
    a, b = r.integers(0, 120, size=(M, K)).astype(np.uint8), (r.integers(0, 120, size=(N, K)) + 128 * r.integers(0, 2, size=(N, K))).astype(np.uint8)
    sa, sb = r.integers(108, 114, size=(M, 2)).astype(np.uint8), r.random((2, 2)).astype(np.float32)
    mag, out = dense.gemm_fp8(a, sa, b, sb)

    def value(c):
        c = int(c)
        e, f = (c >> 3) & 15, c & 7
        v = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        return -v if c & 128 else v
    for m, n in ((0, 0), (1, 127), (2, 128), (0, 129)):
        t = [value(a[m, k]) * 2.0 ** (int(sa[m, k // 128]) - 127) * value(b[n, k]) * float(sb[n // 128, k // 128]) for k in range(K)]
        assert abs(out[m, n] - np.sum(t)) <= 1e-12 * mag[m, n] and abs(mag[m, n] - np.abs(t).sum()) <= 1e-12 * mag[m, n]
    # the gated form's up rows have blocks of their own, counted from their first row
    w13, s13 = np.concatenate([b, b[::-1]]), np.concatenate([sb, 2 * sb])
    g, u, _, _, h = dense.glu_fp8(a, sa, w13, s13)
    assert np.allclose(g, out) and np.allclose(u, dense.gemm_fp8(a, sa, np.ascontiguousarray(b[::-1]), 2 * sb)[1])
    assert np.allclose(h, g / (1 + np.exp(-g)) * u)
    assert np.isnan(dense.e8m0([255])[0]) and dense.e8m0([127, 126]).tolist() == [1.0, 0.5]
