"""The FP8 products with a scale for each block of 128, and drawing a token, as cases that can be timed.

Three operators: the e4m3 matrix product whose rows carry a power of two for
every 128 columns and whose weights an fp32 scale for every 128 x 128 block
(gemm_fp8), the gated form of a shared expert (glu_fp8), and the draw of one
token per row of logits with temperature, top-k, top-p and min-p from given
random numbers (sample). With `own` false, run() computes them in plain torch
operations; with `own` true it calls the framework.
"""
import numpy as np
import torch

own = False

BLOCK = 128
MOST_FLOPS = 2.0 * 4096 * 8192 * 8192
MOST_WEIGHTS = 131072 * 2048
MOST_LOGITS = 256 * 131072


def listed():
    return [
        # a square projection at decode, one token: the weights are read once
        {"name": "gemm-1x2048x2048", "op": "gemm", "M": 1, "N": 2048, "K": 2048, "bias": False, "add": False, "f32": False},
        # a shared expert's down projection at decode, added to the routed experts' output
        {"name": "gemm-32x2048x512-add", "op": "gemm", "M": 32, "N": 2048, "K": 512, "bias": False, "add": True, "f32": False},
        # a ragged prompt into a head of odd width: no size a multiple of a tile or block, fp32 out
        {"name": "gemm-333x1000x4112-f32", "op": "gemm", "M": 333, "N": 1000, "K": 4112, "bias": True, "add": False, "f32": True},
        # the logits of a decode batch over a large vocabulary
        {"name": "gemm-8x131072x2048-f32", "op": "gemm", "M": 8, "N": 131072, "K": 2048, "bias": False, "add": False, "f32": True},
        # the module-batched layer's 16k tokens through a square projection
        {"name": "gemm-16384x2048x2048", "op": "gemm", "M": 16384, "N": 2048, "K": 2048, "bias": False, "add": False, "f32": False},
        # a large dense projection
        {"name": "gemm-4096x8192x8192", "op": "gemm", "M": 4096, "N": 8192, "K": 8192, "bias": False, "add": False, "f32": False},
        # a shared expert's gate and up projections at decode
        {"name": "glu-8x512x2048", "op": "glu", "M": 8, "I": 512, "K": 2048},
        # ... and module-batched
        {"name": "glu-16384x512x2048", "op": "glu", "M": 16384, "I": 512, "K": 2048},
        # one request's next token, over a large vocabulary, with the usual filters
        {"name": "sample-1x131072-f32", "op": "sample", "B": 1, "V": 131072, "bf16": False, "t": True, "k": True, "p": True, "m": False},
        # a decode batch over a vocabulary of odd size; bf16 logits, many of them equal
        {"name": "sample-32x50021-bf16", "op": "sample", "B": 32, "V": 50021, "bf16": True, "t": True, "k": False, "p": True, "m": True},
        # temperature alone: every token can be drawn
        {"name": "sample-64x32768-f32-all", "op": "sample", "B": 64, "V": 32768, "bf16": False, "t": True, "k": False, "p": False, "m": False},
        # a large batch of requests, every filter
        {"name": "sample-256x131072-f32", "op": "sample", "B": 256, "V": 131072, "bf16": False, "t": True, "k": True, "p": True, "m": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "glu", "sample", "sample"])
    if op == "sample":
        V = _log(rng, 512, 196608)
        if rng.random() < 0.5:
            V = max(512, V // 128 * 128)
        B = max(1, min(_log(rng, 1, 512), MOST_LOGITS // V))
        return {"op": "sample", "B": B, "V": V, "bf16": rng.random() < 0.4, "t": rng.random() < 0.8, "k": rng.random() < 0.5,
                "p": rng.random() < 0.6, "m": rng.random() < 0.4}
    M = _log(rng, 1, 16384)
    K = max(16, _log(rng, 128, 8192) // 16 * 16)
    if rng.random() < 0.7:
        K = max(128, K // 128 * 128)
    if op == "gemm":
        N = _log(rng, 64, 131072)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        N = max(64, min(N, MOST_WEIGHTS // K))
        M = max(1, min(M, int(MOST_FLOPS / 2 / N / K)))
        return {"op": "gemm", "M": M, "N": N, "K": K, "bias": rng.random() < 0.4, "add": rng.random() < 0.4, "f32": rng.random() < 0.3}
    I = _log(rng, 64, 4096)
    if rng.random() < 0.7:
        I = max(64, I // 64 * 64)
    M = max(1, min(M, int(MOST_FLOPS / 4 / I / K)))
    return {"op": "glu", "M": M, "I": I, "K": K}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": dict(case)}

    def rand(*size):
        return torch.rand(*size, device=dev, generator=g)

    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        # a broad bulk and a few favoured tokens, as a head gives them
        z = 2.2 * torch.randn(B, V, device=dev, generator=g)
        few = torch.randint(V, (B, 24), device=dev, generator=g)
        z.scatter_add_(1, few, 4 + 8 * rand(B, 24))
        s["logits"] = z.to(torch.bfloat16) if case["bf16"] else z
        s["u"] = rand(B)
        # every row a request of its own: some greedy, some without a filter
        t = 0.4 + rand(B)
        s["t"] = torch.where(rand(B) < 0.1, torch.zeros_like(t), t) if case["t"] else None
        k = torch.exp(rand(B) * 7).to(torch.int32)
        s["k"] = torch.where(rand(B) < 0.2, torch.zeros_like(k), k) if case["k"] else None
        s["p"] = torch.where(rand(B) < 0.1, torch.ones(B, device=dev), 0.7 + 0.3 * rand(B)) if case["p"] else None
        s["m"] = 0.1 * rand(B) if case["m"] else None
        return s
    M, K = case["M"], case["K"]

    def codes(rows):
        # rows quantized by the largest of each 128 values, which is near 2.6 deviations
        c = torch.randn(rows, K, device=dev, generator=g).mul_(110.0).clamp_(-448, 448)
        return c.to(torch.float8_e4m3fn).view(torch.uint8)

    s["a"] = codes(M)
    s["sa"] = torch.randint(118, 122, (M, _blocks(K)), device=dev, generator=g, dtype=torch.uint8)
    if case["op"] == "glu":
        I = case["I"]
        s["b"] = codes(2 * I)
        blocks = 2 * _blocks(I)
    else:
        N = case["N"]
        s["b"] = codes(N)
        blocks = _blocks(N)
        out = torch.float32 if case["f32"] else torch.bfloat16
        s["out"] = out
        s["bias"] = torch.randn(N, device=dev, generator=g) if case["bias"] else None
        s["add"] = torch.randn(M, N, device=dev, generator=g).to(out) if case["add"] else None
    s["sb"] = 0.01 / K ** 0.5 * torch.exp(0.3 * torch.randn(blocks, _blocks(K), device=dev, generator=g))
    return s


def _columns(scale, K):
    """A scale for each 128 columns, written out for every column."""
    return scale.repeat_interleave(BLOCK, dim=1)[:, :K]


def _weights(codes, scale):
    """e4m3 codes of a weight matrix -> fp32 values."""
    rows, K = codes.shape
    return codes.view(torch.float8_e4m3fn).float() * _columns(scale, K).repeat_interleave(BLOCK, dim=0)[:rows]


def _plain_sample(s):
    logits = s["logits"]
    B, V = logits.shape
    # weights, sums and borders in 64 bits: a sum decides which token is drawn
    z, order = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    z = z.double()
    one = torch.ones(B, 1, dtype=torch.float64, device=z.device)
    t = one if s["t"] is None else s["t"].double()[:, None]
    greedy = t == 0
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, one, t))
    place = torch.arange(V, device=z.device)[None, :]
    keep = torch.where(greedy, place < 1, place < V)
    if s["k"] is not None:
        k = s["k"][:, None]
        keep = keep & ((place < k) | (k <= 0))
    if s["p"] is not None:
        kept = torch.where(keep, w, 0.0)
        before = torch.cumsum(kept, dim=1) - kept
        keep = keep & ((before < s["p"].double()[:, None] * kept.sum(dim=1, keepdim=True)) | (place < 1))
    if s["m"] is not None:
        keep = keep & (w >= s["m"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    sums = torch.cumsum(w, dim=1)
    total = sums[:, -1:]
    ids = (sums > s["u"].double()[:, None] * total).to(torch.int32).argmax(dim=1, keepdim=True)
    return ids[:, 0].to(torch.int32), (w.gather(1, ids) / total)[:, 0].float()


def _run_plain(s):
    c = s["case"]
    if c["op"] == "sample":
        return _plain_sample(s)
    K = c["K"]
    a = s["a"].view(torch.float8_e4m3fn).float() * _columns(torch.exp2(s["sa"].float() - 127), K)
    if c["op"] == "glu":
        I, half = c["I"], _blocks(c["I"])
        gate = torch.matmul(a, _weights(s["b"][:I], s["sb"][:half]).t())
        up = torch.matmul(a, _weights(s["b"][I:], s["sb"][half:]).t())
        return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    p = torch.matmul(a, _weights(s["b"], s["sb"]).t())
    if c["bias"]:
        p = p + s["bias"]
    if c["add"]:
        p = p + s["add"].float()
    return p.to(s["out"])


def _run_own(s):
    import moe_expert_layer_topk_amd as moe
    c = s["case"]
    if c["op"] == "sample":
        ids, p, _ = moe.sample(s["logits"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
        return ids, p
    if c["op"] == "glu":
        return moe.glu_fp8(s["a"], s["sa"], s["b"], s["sb"])
    return moe.gemm_fp8(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], add=s["add"], out_dtype=s["out"])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    if case["op"] == "sample":
        n = case["B"] * case["V"]
        return {"bytes": n * (2 if case["bf16"] else 4) + 28 * case["B"], "flops": 4 * n}
    M, K = case["M"], case["K"]
    kb = _blocks(K)
    if case["op"] == "glu":
        I = case["I"]
        return {"bytes": M * (K + kb) + 2 * I * K + 8 * _blocks(I) * kb + 2 * M * I, "flops": 4.0 * M * I * K}
    N = case["N"]
    o = M * N * (4 if case["f32"] else 2)
    return {"bytes": M * (K + kb) + N * K + 4 * _blocks(N) * kb + (4 * N if case["bias"] else 0) + o + (o if case["add"] else 0),
            "flops": 2.0 * M * N * K}


def _e4m3(codes):
    """Values of e4m3 codes in fp64, from the fields: 1 sign, 4 exponent (bias 7) and 3 fraction bits."""
    c = torch.arange(256, dtype=torch.float64)
    e, f = torch.floor(c / 8) % 16, c % 8
    v = torch.where(e > 0, (8 + f) / 8 * 2.0 ** (e - 7), f / 8 * 2.0 ** -6)
    v = torch.where(c >= 128, -v, v)
    return v.to(codes.device)[codes.long()]


def _exact_sample(s):
    """Row by row on the host: the tokens in order, the filters as lengths of that order, the sums over kept tokens."""
    logits = s["logits"].double().cpu().numpy()
    B, V = logits.shape
    host = {n: None if s[n] is None else s[n].double().cpu().numpy() for n in ("u", "t", "k", "p", "m")}
    ids, probs = np.zeros(B, np.int32), np.zeros(B)
    for b in range(B):
        order = np.argsort(-logits[b], kind="stable")
        t = 1.0 if host["t"] is None else host["t"][b]
        if t == 0:
            ids[b], probs[b] = order[0], 1.0
            continue
        w = np.exp((logits[b][order] - logits[b][order[0]]) / t)
        n = V
        if host["k"] is not None and host["k"][b] > 0:
            n = min(n, int(host["k"][b]))
        if host["p"] is not None:
            ends = np.cumsum(w[:n])
            n = 1 + int(np.searchsorted(ends[:-1], host["p"][b] * ends[-1], side="left"))
        if host["m"] is not None:
            n = min(n, int(np.searchsorted(-w, -host["m"][b], side="right")))
        kept = np.sort(order[:n])
        weight = np.exp((logits[b][kept] - logits[b][order[0]]) / t)
        ends = np.cumsum(weight)
        at = min(int(np.searchsorted(ends, host["u"][b] * ends[-1], side="right")), n - 1)
        ids[b], probs[b] = kept[at], weight[at] / ends[-1]
    return torch.from_numpy(ids).to(s["logits"].device), torch.from_numpy(probs).to(s["logits"].device)


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "sample":
        return _exact_sample(s)
    K, kb = case["K"], _blocks(case["K"])

    def product(b, sb):
        out = torch.zeros(case["M"], b.shape[0], dtype=f, device=b.device)
        for n in range(0, b.shape[0], 16384):                # (fp64 weights of a part of the columns at a time)
            v = _e4m3(b[n:n + 16384])
            rows = torch.arange(n, n + v.shape[0], device=b.device) // BLOCK
            for j in range(kb):
                v[:, j * BLOCK:(j + 1) * BLOCK] *= sb[rows, j].to(f)[:, None]
            out[:, n:n + v.shape[0]] = torch.mm(a, v.t().contiguous())
        return out

    a = _e4m3(s["a"])
    for j in range(kb):
        a[:, j * BLOCK:(j + 1) * BLOCK] *= torch.pow(2.0, s["sa"][:, j].to(f) - 127)[:, None]
    if case["op"] == "glu":
        I, half = case["I"], _blocks(case["I"])
        gate, up = product(s["b"][:I], s["sb"][:half]), product(s["b"][I:], s["sb"][half:])
        return gate * torch.sigmoid(gate) * up
    out = product(s["b"], s["sb"])
    if case["bias"]:
        out += s["bias"].to(f)
    if case["add"]:
        out += s["add"].to(f)
    return out
