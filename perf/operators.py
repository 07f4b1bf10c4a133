"""The dense 8-bit operators around the expert layer, as cases that can be timed.

Four operators: the residual addition with RMS norm and 8-bit output (norm),
the row quantizer (quant_rows), the int8 matrix product with a scale per token
and channel (gemm_i8), and the gated int8 product of a shared expert (glu_i8).
With `own` false, run() computes them in plain fp32 torch operations; with
`own` true it calls the framework.
"""
import torch

own = False

FLOOR = 2.0 ** -100      # a row maximum below this is quantized as if it were this
EPS = 1e-6
MOST_FLOPS = 2.0 * 4096 * 8192 * 8192
MOST_ELEMS = 16384 * 2048


def listed():
    return [
        # one token of a decode step entering the block: int8 rows for the shared expert, bf16 rows for the router
        {"name": "norm-1x2048-i8", "op": "norm", "T": 1, "H": 2048, "res": True, "w": True, "q": "i8", "y": True},
        # a prefill batch whose norm feeds the FP8 expert layer
        {"name": "norm-4096x2048-fp8", "op": "norm", "T": 4096, "H": 2048, "res": True, "w": True, "q": "fp8", "y": True},
        # the module-batched layer's 16k tokens
        {"name": "norm-16384x2048-i8", "op": "norm", "T": 16384, "H": 2048, "res": True, "w": True, "q": "i8", "y": True},
        # h rows of a shared expert's down projection, decode
        {"name": "quant-32x768", "op": "quant", "T": 32, "H": 768},
        # ... and module-batched
        {"name": "quant-16384x512", "op": "quant", "T": 16384, "H": 512},
        # a square projection at decode, one token: the weights are read once
        {"name": "gemm-1x2048x2048", "op": "gemm", "M": 1, "N": 2048, "K": 2048, "bias": False, "add": False, "f32": False},
        # a shared expert's down projection at decode, added to the routed experts' output
        {"name": "gemm-32x2048x512-add", "op": "gemm", "M": 32, "N": 2048, "K": 512, "bias": False, "add": True, "f32": False},
        # a ragged prompt into a head of odd width: no size a multiple of a tile, fp32 out
        {"name": "gemm-333x1000x4112-f32", "op": "gemm", "M": 333, "N": 1000, "K": 4112, "bias": True, "add": False, "f32": True},
        # the module-batched layer's 16k tokens through a square projection
        {"name": "gemm-16384x2048x2048", "op": "gemm", "M": 16384, "N": 2048, "K": 2048, "bias": False, "add": False, "f32": False},
        # a large dense projection
        {"name": "gemm-4096x8192x8192", "op": "gemm", "M": 4096, "N": 8192, "K": 8192, "bias": False, "add": False, "f32": False},
        # a shared expert's gate and up projections at decode
        {"name": "glu-8x512x2048", "op": "glu", "M": 8, "I": 512, "K": 2048},
        # ... and module-batched
        {"name": "glu-16384x512x2048", "op": "glu", "M": 16384, "I": 512, "K": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "glu"])
    if op in ("norm", "quant"):
        T = _log(rng, 1, 16384)
        H = _log(rng, 64, 8192)
        case = {"op": op, "T": T, "H": H}
        if op == "norm":
            q = rng.choice(["none", "i8", "fp8"])
            if q == "fp8":
                H = max(128, H // 128 * 128)
            case.update({"H": H, "res": rng.random() < 0.7, "w": rng.random() < 0.8, "q": q,
                         "y": q == "none" or rng.random() < 0.6})
        elif rng.random() < 0.6:
            case["H"] = max(64, H // 64 * 64)
        case["T"] = max(1, min(T, MOST_ELEMS // case["H"]))
        return case
    M = _log(rng, 1, 16384)
    K = max(16, _log(rng, 128, 8192) // 16 * 16)
    if rng.random() < 0.6:
        K = max(128, K // 128 * 128)
    if op == "gemm":
        N = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        M = max(1, min(M, int(MOST_FLOPS / 2 / N / K)))
        return {"op": "gemm", "M": M, "N": N, "K": K, "bias": rng.random() < 0.4, "add": rng.random() < 0.4,
                "f32": rng.random() < 0.3}
    I = _log(rng, 64, 4096)
    if rng.random() < 0.7:
        I = max(64, I // 64 * 64)
    M = max(1, min(M, int(MOST_FLOPS / 4 / I / K)))
    return {"op": "glu", "M": M, "I": I, "K": K}


def _rows(case):
    """Rows of token states: normal values, some channels far larger than the rest, as hidden states have them."""
    return case["T"], case["H"]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["op"] in ("norm", "quant"):
        T, H = _rows(case)
        chan = torch.exp(0.7 * torch.randn(H, device=dev, generator=g))
        s["x"] = (torch.randn(T, H, device=dev, generator=g) * chan).to(torch.bfloat16)
        if case["op"] == "norm":
            s["res"] = (2 * torch.randn(T, H, device=dev, generator=g) * chan).to(torch.bfloat16) if case["res"] else None
            s["w"] = 1 + 0.2 * torch.randn(H, device=dev, generator=g) if case["w"] else None
        return s
    M, K = case["M"], case["K"]
    N = case["N"] if case["op"] == "gemm" else 2 * case["I"]

    def codes(rows, spread):
        c = torch.randn(rows, K, device=dev, generator=g).mul_(spread).round_().clamp_(-127, 127)
        return c.to(torch.int8)

    # rows quantized by their largest value: normal rows of some thousand values have it near 3.6 deviations
    s["a"], s["sa"] = codes(M, 35.0), 0.028 * torch.exp(0.3 * torch.randn(M, device=dev, generator=g))
    s["b"], s["sb"] = codes(N, 35.0), 0.028 / K ** 0.5 * torch.exp(0.3 * torch.randn(N, device=dev, generator=g))
    if case["op"] == "gemm":
        out = torch.float32 if case["f32"] else torch.bfloat16
        s["out"] = out
        s["bias"] = torch.randn(N, device=dev, generator=g) if case["bias"] else None
        s["add"] = torch.randn(M, N, device=dev, generator=g).to(out) if case["add"] else None
    return s


def _plain_i8(v):
    """Rows of fp32 values -> (the values their int8 codes stand for, in bf16; fp32 scales)."""
    m = v.abs().amax(dim=1, keepdim=True).clamp_min(FLOOR)
    code = torch.round(v * (127.0 / m)).clamp(-127, 127)
    scale = m / 127.0
    return (code * scale).to(torch.bfloat16), scale[:, 0]


def _plain_fp8(v):
    """Rows of fp32 values -> e4m3 codes and one power-of-two scale per 128 columns."""
    T, H = v.shape
    g = v.view(T, H // 128, 128)
    m = g.abs().amax(dim=2, keepdim=True)
    # smallest s with m <= 448 2^s = 0.875 2^(9 + s), m = f 2^e with f in [0.5, 1)
    f, e = torch.frexp(m)
    s = torch.where(m > 0, e - 9 + (f > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(-127, 127)
    codes = torch.ldexp(g, -s).to(torch.float8_e4m3fn).view(T, H)
    return codes, (s + 127).to(torch.uint8)[:, :, 0].contiguous().view(torch.float8_e8m0fnu)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quant":
        return _plain_i8(s["x"].float())
    if c["op"] == "norm":
        v = s["x"].float()
        if c["res"]:
            v = v + s["res"].float()
        y = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
        if c["w"]:
            y = y * s["w"]
        out = {}
        if c["y"]:
            out["y"] = y.to(torch.bfloat16)
        if c["res"]:
            out["sum"] = v.to(torch.bfloat16)
        if c["q"] == "i8":
            out["q"], out["scale"] = _plain_i8(y)
        elif c["q"] == "fp8":
            out["q"], out["scale"] = _plain_fp8(y)
        return out
    p = torch.matmul(s["a"].float(), s["b"].float().t()) * s["sa"][:, None] * s["sb"][None, :]
    if c["op"] == "glu":
        gate, up = p[:, :c["I"]], p[:, c["I"]:]
        return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    if c["bias"]:
        p = p + s["bias"]
    if c["add"]:
        p = p + s["add"].float()
    return p.to(s["out"])


def _run_own(s):
    import moe_expert_layer_topk_amd as moe
    c = s["case"]
    if c["op"] == "quant":
        codes, scale = moe.quant_rows(s["x"])
        return moe.dequant_rows(codes, scale), scale
    if c["op"] == "norm":
        mode = {"none": moe.Q_NONE, "i8": moe.Q_I8_ROW, "fp8": moe.Q_FP8_G128_POW2}[c["q"]]
        y, total, codes, scale = moe.norm(s["x"], s["w"], EPS, res=s["res"], q_mode=mode, with_y=c["y"])
        out = {}
        if c["y"]:
            out["y"] = y
        if c["res"]:
            out["sum"] = total
        if c["q"] == "i8":
            out["q"], out["scale"] = moe.dequant_rows(codes, scale), scale
        elif c["q"] == "fp8":
            out["q"], out["scale"] = codes.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)
        return out
    if c["op"] == "glu":
        return moe.glu_i8(s["a"], s["sa"], s["b"], s["sb"])
    return moe.gemm_i8(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], add=s["add"], out_dtype=s["out"])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    if case["op"] in ("norm", "quant"):
        T, H = _rows(case)
        n = T * H
        if case["op"] == "quant":
            return {"bytes": 3 * n + 4 * T, "flops": 4 * n}
        size = 2 * n + (4 * n if case["res"] else 0) + (2 * n if case["y"] else 0) + (4 * H if case["w"] else 0)
        if case["q"] == "i8":
            size += n + 4 * T
        elif case["q"] == "fp8":
            size += n + n // 128
        return {"bytes": size, "flops": 8 * n}
    M, K = case["M"], case["K"]
    if case["op"] == "glu":
        I = case["I"]
        return {"bytes": M * K + 2 * I * K + 4 * M + 8 * I + 2 * M * I, "flops": 4.0 * M * I * K}
    N = case["N"]
    o = M * N * (4 if case["f32"] else 2)
    return {"bytes": M * K + N * K + 4 * M + 4 * N + (4 * N if case["bias"] else 0) + o + (o if case["add"] else 0),
            "flops": 2.0 * M * N * K}


def _e4m3_value(v):
    """The e4m3 value nearest to each |v| <= 448 (ties to even), in fp64: steps of 2^(e - 3) with e = floor(log2|v|) >= -6."""
    e = torch.frexp(v)[1].to(torch.float64) - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    """The operators' definitions in 64 bits: what 8 bits hold is rounded, the rest is not."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] in ("norm", "quant"):
        x = s["x"].to(f)

        def i8(v):
            m = torch.maximum(v.abs().max(dim=1).values, torch.tensor(FLOOR, dtype=f, device=v.device))[:, None]
            return torch.round(v * 127 / m) * m / 127, m[:, 0] / 127

        if case["op"] == "quant":
            return i8(x)
        total = x + s["res"].to(f) if case["res"] else x
        y = total / torch.sqrt(total.pow(2).sum(dim=1, keepdim=True) / case["H"] + EPS)
        if case["w"]:
            y = y * s["w"].to(f)
        out = {}
        if case["y"]:
            out["y"] = y
        if case["res"]:
            out["sum"] = total
        if case["q"] == "i8":
            out["q"], out["scale"] = i8(y)
        elif case["q"] == "fp8":
            groups = y.reshape(y.shape[0], -1, 128)
            m = groups.abs().amax(dim=2, keepdim=True)
            two = torch.exp2(torch.ceil(torch.log2(m / 448)).clamp(-127, 127))
            two = torch.where(m > 0, two, torch.ones_like(two))
            out["q"] = _e4m3_value(groups / two).reshape(y.shape)
            out["scale"] = two[:, :, 0]
        return out
    a = s["a"].to(f) * s["sa"].to(f)[:, None]
    b = s["b"].to(f) * s["sb"].to(f)[:, None]
    if case["op"] == "glu":
        I = case["I"]
        gate = torch.mm(a, b[:I].t().contiguous())
        up = torch.mm(a, b[I:].t().contiguous())
        return gate * torch.sigmoid(gate) * up
    out = torch.mm(a, b.t().contiguous())
    if case["bias"]:
        out += s["bias"].to(f)
    if case["add"]:
        out += s["add"].to(f)
    return out
