"""moe_sample where a parameter stands at its border: top_p of zero and less beside
min_p among equal logits, top_k up to int32's largest. Whole numbers, but for what
is compared with the oracle, where decisions and tolerances are those of
test_gpu_sample.py.
"""
import numpy as np
import pytest

import moe_expert_layer_topk_amd as moe
from test_gpu_sample import _dev, _say
from test_gpu_sample_edges import _against_oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,ties", [(5000, 5000), (8192, 8192), (9000, 9000), (50021, 300), (131072, 700)])
@pytest.mark.parametrize("bf16", [False, True])
def test_top_p_of_nothing_keeps_the_first_token(gpu, V, ties, bf16):
    """However many others have its logit and min_p would keep (more than a chunk may list)."""
    import torch
    f = np.float32
    r = np.random.default_rng([41, V])
    B = 6
    l = (r.normal(size=(B, V)) * 0.3).astype(f)
    at = min(4096, V - ties)
    l[:, at:at + ties] = 4.0
    l = torch.from_numpy(l).to(torch.bfloat16 if bf16 else torch.float32).to(gpu)
    u = r.random(B).astype(f)
    for pp, mp in ((0.0, 0.1), (0.0, 1.0), (-1.0, 0.5), (0.0, 1e-6), (1e-45, 0.1), (1e-9, 0.1), (0.0, None), (-np.inf, None)):
        for k in (None, 0, V + 5, 2000):
            _say(f"[top_p of nothing] V={V} {ties} equal, p={pp} m={mp} k={k}")
            par = [None, None if k is None else np.full(B, k, np.int32), np.full(B, pp, f), None if mp is None else np.full(B, mp, f)]
            ids, p, _ = moe.sample(l, _dev(u, gpu), *(_dev(v, gpu) for v in par))
            assert ids.tolist() == [at] * B and p.tolist() == [1.0] * B


@pytest.mark.parametrize("V", [60, 700, 4096, 4097, 131072])
def test_top_k_up_to_the_largest_int(gpu, V):
    """As many as the row has and any number above are the same call."""
    import torch
    f = np.float32
    r = np.random.default_rng([42, V])
    B = 8
    l = (r.normal(size=(B, V)) * np.array([0.01, 0.5, 2, 5] * 2)[:, None]).astype(f)
    u, t = r.random(B).astype(f), (0.5 + r.random(B)).astype(f)
    for pp, mp in ((None, None), (0.9, None), (None, 0.02), (0.95, 0.001)):
        rest = [None if pp is None else np.full(B, pp, f), None if mp is None else np.full(B, mp, f)]
        _say(f"[top_k] V={V} p={pp} m={mp}")
        want = moe.sample(*(_dev(v, gpu) for v in (l, u, t, np.full(B, V, np.int32), *rest)))
        for k in (V + 1, 1 << 20, 2 ** 30 - 33, 2 ** 30 - 32, 2 ** 30, 2 ** 31 - 1):
            got = moe.sample(*(_dev(v, gpu) for v in (l, u, t, np.full(B, k, np.int32), *rest)))
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), k
        _against_oracle(gpu, l, u, [t, np.full(B, 2 ** 31 - 1, np.int32), *rest])
