"""Cases of the operators that join the products of a transformer block with mixture-of-experts layers, in the forms a program
calls them:

norm      root-mean-square norm of a row and its residual, with its output as it is or as e4m3 codes with a scale per 128 (fp32
          or a power of two), the left operand of the FP8 products; with its gradient
epilogue  block-scaled FP8 product, then bias, activation and residual
dact      gradient of that epilogue: of the product (bf16, and as e4m3 codes with scales) and of the bias
experts   the experts of a mixture-of-experts layer for a few tokens: gate and up projection, SiLU(gate) * up, down projection,
          weighted sum; weights in block-scaled FP8 or in microscaled 4-bit floats

Each has a plain form in elementary 32-bit torch operations, the framework's own call (``own``), and its definition in 64
bits (``exact``)."""

import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # one decode step of one sequence: the norm before the router, latency
        {"name": "norm_token", "op": "norm", "M": 1, "K": 7168, "dtype": "bf16", "residual": True, "out": "fp8", "grad": False},
        # a prefill batch: residual stream in, operand of the next product out
        {"name": "norm_prefill", "op": "norm", "M": 16384, "K": 7168, "dtype": "bf16", "residual": True, "out": "fp8", "grad": False},
        # a ragged batch of an fp32 residual stream, power-of-two scales
        {"name": "norm_ragged", "op": "norm", "M": 1021, "K": 2048, "dtype": "f32", "residual": True, "out": "ue8m0", "grad": False},
        # a training step, forward and backward
        {"name": "norm_train", "op": "norm", "M": 8192, "K": 4096, "dtype": "bf16", "residual": True, "out": "y", "grad": True},
        # decode: a small batch against one weight, bias and activation
        {"name": "epilogue_decode", "op": "epilogue", "M": 64, "N": 4096, "K": 7168, "act": "silu", "bias": True, "residual": False, "pre": False},
        # prefill: projection back into the residual stream, an odd number of rows
        {"name": "epilogue_prefill", "op": "epilogue", "M": 4095, "N": 7168, "K": 2048, "act": "none", "bias": True, "residual": True, "pre": False},
        # training forward: what the backward pass needs is kept
        {"name": "epilogue_train", "op": "epilogue", "M": 4096, "N": 4096, "K": 7168, "act": "gelu", "bias": True, "residual": False, "pre": True},
        # training backward: gradient of the product, quantised for the next one, and of the bias
        {"name": "dact_train", "op": "dact", "M": 4096, "N": 4096, "act": "gelu", "bias": True, "quant": True},
        # one token through a small layer: latency
        {"name": "experts_small", "op": "experts", "T": 1, "k": 4, "E": 16, "first": 0, "G": 16, "H": 1024, "I": 512, "fmt": "fp8", "pad": 0.0},
        # one token through a large layer whose experts are all here
        {"name": "experts_token", "op": "experts", "T": 1, "k": 8, "E": 32, "first": 0, "G": 32, "H": 7168, "I": 2048, "fmt": "fp8", "pad": 0.0},
        # a decode step on a GPU that holds 32 of 256 experts, some of the batch being padding
        {"name": "experts_batch", "op": "experts", "T": 48, "k": 8, "E": 256, "first": 64, "G": 32, "H": 7168, "I": 2048, "fmt": "mxfp4", "pad": 0.1},
        # a full batch over few experts: every expert has several tokens
        {"name": "experts_full", "op": "experts", "T": 64, "k": 2, "E": 8, "first": 0, "G": 8, "H": 4096, "I": 2048, "fmt": "fp8", "pad": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    """A size, a multiple of `step` from lo * step to hi * step, even over its logarithm."""
    return step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "epilogue", "epilogue", "dact", "experts", "experts", "experts"])
    if op == "norm":
        out = rng.choice(["fp8", "fp8", "ue8m0", "y"])
        K = _log(rng, 8, 900, 8) if out == "y" else _log(rng, 1, 56, 128)
        return {"op": op, "M": _log(rng, 1, 8192), "K": K, "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.7,
                "out": out, "grad": out == "y" and rng.random() < 0.7}
    if op == "epilogue":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 8, 256, 16), "K": _log(rng, 2, 56, 128),
                "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.5, "pre": rng.random() < 0.4}
    if op == "dact":
        quant = rng.random() < 0.6
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 1, 32, 128) if quant else _log(rng, 8, 256, 16),
                "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.7, "quant": quant}
    E = rng.choice([8, 16, 60, 64, 128, 256])
    G = min(32, rng.choice([E, max(1, E // 2), max(1, E // 8)]))
    return {"op": op, "T": _log(rng, 1, 64), "k": rng.randint(1, min(E, 8)), "E": E, "first": rng.randint(0, E - G), "G": G,
            "H": _log(rng, 2, 40, 128), "I": _log(rng, 1, 16, 128), "fmt": rng.choice(["fp8", "mxfp4"]), "pad": rng.choice([0.0, 0.0, 0.2])}


# ---- what a program has in hand


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(shape, g, dtype=torch.float32):
    """Unit normal values, one in a thousand twenty times as large."""
    x = torch.randn(shape, device=DEV, generator=g)
    return torch.where(torch.rand(shape, device=DEV, generator=g) < 1e-3, 20 * x, x).to(dtype)


def _e4m3_operand(rows, K, g):
    """Codes [rows, K] and scales [K / 128, rows] of activations: a row's largest of 128 is 448."""
    x = _activations((rows, K), g).reshape(rows, K // 128, 128)
    s = x.abs().amax(-1) / 448
    return (x / s[..., None]).to(FP8).view(torch.uint8).reshape(rows, K), s.t().contiguous()


def _e4m3_weight(N, K, g):
    """Codes [N, K] and scales [ceil(N / 128), K / 128] of a weight: normal values of about 1 / sqrt(K), a block's largest near 448."""
    q = (110 * torch.randn(N, K, device=DEV, generator=g)).clamp(-448, 448).to(FP8).view(torch.uint8)
    s = (0.8 + 0.4 * torch.rand((N + 127) // 128, K // 128, device=DEV, generator=g)) / (110 * math.sqrt(K))
    return q, s


def _fp4_grid():
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)


def _fp4_weight(N, K, g):
    """Packed codes [N, K / 2] (low nibble first) and scale words [K / 128, N] (the codes of four blocks of 32, 2^(c - 127))."""
    x = torch.randn(N, K // 32, 32, device=DEV, generator=g) / math.sqrt(K)
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.75, e - 3, e - 2)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    c = (torch.bucketize(torch.ldexp(x.abs(), -e[..., None]), mid) + 8 * torch.signbit(x)).to(torch.uint8).reshape(N, K // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), (e + 127).to(torch.uint8).contiguous().view(torch.int32).t().contiguous()


def prepare(case, seed):
    op = case["op"]
    s = dict(case)
    g = _gen(seed)
    if op == "norm":
        M, K = case["M"], case["K"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = _activations((M, K), g, dt)
        s["res"] = _activations((M, K), g, dt) if case["residual"] else None
        s["weight"] = (1 + 0.1 * torch.randn(K, device=DEV, generator=g)).to(dt)
        s["h"] = torch.empty(M, K, dtype=dt, device=DEV) if case["residual"] else None
        s["y"] = torch.empty(M, K, dtype=dt, device=DEV) if case["out"] == "y" else None
        s["q"] = torch.empty(M, K, dtype=torch.uint8, device=DEV) if case["out"] != "y" else None
        s["sf"] = {"fp8": lambda: torch.empty(K // 128, M, device=DEV),
                   "ue8m0": lambda: torch.empty((K + 511) // 512, M, dtype=torch.int32, device=DEV), "y": lambda: None}[case["out"]]()
        s["rstd"] = torch.empty(M, device=DEV)
        if case["grad"]:
            s["dy"], s["dh"] = (torch.randn(M, K, device=DEV, generator=g).to(dt) for _ in range(2))
            s["dx"], s["dw"] = torch.empty(M, K, dtype=dt, device=DEV), torch.empty(K, device=DEV)
            s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    elif op == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["sfa"] = _e4m3_operand(M, K, g)
        s["B"], s["sfb"] = _e4m3_weight(N, K, g)
        s["b"] = 0.5 * torch.randn(N, device=DEV, generator=g) if case["bias"] else None
        s["res"] = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16) if case["residual"] else None
        s["Z"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV) if case["pre"] else None
        s["D"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    elif op == "dact":
        M, N = case["M"], case["N"]
        s["dy"] = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16)
        s["Z"] = (1.1 * torch.randn(M, N, device=DEV, generator=g)).to(torch.bfloat16) if case["act"] != "none" else None
        s["dz"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        s["q"] = torch.empty(M, N, dtype=torch.uint8, device=DEV) if case["quant"] else None
        s["sf"] = torch.empty(N // 128, M, device=DEV) if case["quant"] else None
        s["db"] = torch.empty(N, device=DEV) if case["bias"] else None
        s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    else:
        T, k, E, G, H, I = (case[n] for n in ("T", "k", "E", "G", "H", "I"))
        weight = _e4m3_weight if case["fmt"] == "fp8" else _fp4_weight
        w1, w2 = ([weight(n, m, g) for _ in range(G)] for n, m in ((2 * I, H), (H, I)))
        s["w1"], s["s1"] = (torch.stack(t) for t in zip(*w1))
        s["w2"], s["s2"] = (torch.stack(t) for t in zip(*w2))
        s["x"] = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
        popular = 0.5 * torch.randn(E, device=DEV, generator=g)
        logits = popular + torch.randn(T, E, device=DEV, generator=g)
        top = torch.topk(logits, k, dim=1)
        there = torch.rand(T, 1, device=DEV, generator=g) >= case["pad"]
        s["idx"] = torch.where(there, top.indices, -1).int().contiguous()
        s["w"] = torch.where(there, torch.softmax(top.values, 1), 0.0)
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    return s


# ---- one pass


def run(s):
    return (_run_own if own else _run_plain)(s)


def _scales(s):
    """The scales of a quantised output as the values they stand for (power-of-two codes a byte each)."""
    return s["sf"] if s["sf"].dtype is torch.float32 else s["sf"].view(torch.float8_e8m0fnu)


def _run_own(s):
    from moe_grouped_matmul_amd import dg

    op = s["op"]
    if op == "norm":
        dg.dg_rms_norm(s["x"], s["weight"], residual=s["res"], h=s["h"], y=s["y"], q=s["q"], sf=s["sf"], rstd=s["rstd"], eps=EPS)
        out = {"rstd": s["rstd"]}
        if s["residual"]:
            out["h"] = s["h"]
        if s["out"] == "y":
            out["y"] = s["y"]
        else:
            out["q"], out["sf"] = s["q"].view(FP8), _scales(s)
        if s["grad"]:
            dg.dg_rms_norm_bwd(s["dy"], s["h"] if s["residual"] else s["x"], s["weight"], s["rstd"], s["dx"], s["dw"], dh=s["dh"],
                               workspace=s["ws"])
            out["dx"], out["dw"] = s["dx"], s["dw"]
        return out
    if op == "epilogue":
        dg.dg_fp8_gemm_nt_epilogue(s["A"], s["sfa"], s["B"], s["sfb"], s["D"], bias=s["b"], act=s["act"], residual=s["res"], pre=s["Z"],
                                   workspace=s["ws"])
        return {"D": s["D"], "Z": s["Z"]} if s["pre"] else {"D": s["D"]}
    if op == "dact":
        dg.dg_epilogue_bwd(s["dy"], s["dz"], pre=s["Z"], act=s["act"], q=s["q"], sf=s["sf"], dbias=s["db"], workspace=s["ws"])
        out = {"dz": s["dz"]}
        if s["quant"]:
            out["q"], out["sf"] = s["q"].view(FP8), s["sf"]
        if s["bias"]:
            out["db"] = s["db"]
        return out
    call = dg.dg_moe_experts_fp8 if s["fmt"] == "fp8" else dg.dg_moe_experts_mxfp4
    call(s["x"], s["idx"], s["w"], s["w1"], s["s1"], s["w2"], s["s2"], s["out"], first_expert=s["first"], workspace=s["ws"])
    return s["out"]


def _run_plain(s):
    return {"norm": _norm, "epilogue": _epilogue, "dact": _dact, "experts": _experts}[s["op"]](s)


def _to_e4m3(v):
    """fp32 values up to 448 -> the nearest e4m3 values, ties to even."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
    return (torch.round(v / step) * step).to(FP8)


def _quantised(v, kind):
    """Rows of fp32 values -> e4m3 codes [M, K] and scales, as fp32 [K / 128, M] or a power of two's code a byte each."""
    M, K = v.shape
    b = v.reshape(M, K // 128, 128)
    alpha = b.abs().amax(-1) / 448
    alpha = torch.where(alpha > 0, alpha, 1.0)
    if kind == "fp8":
        return _to_e4m3(b / alpha[..., None]).reshape(M, K), alpha.t().contiguous()
    m, e = torch.frexp(alpha)
    e = torch.where(m == 0.5, e - 1, e)
    code = torch.zeros(M, (K + 511) // 512 * 4, dtype=torch.uint8, device=DEV)
    code[:, : K // 128] = (e + 127).to(torch.uint8)
    words = code.view(torch.int32).t().contiguous()
    return _to_e4m3(torch.ldexp(b, -e[..., None])).reshape(M, K), words.view(torch.float8_e8m0fnu)


def _norm(s):
    dt = s["x"].dtype
    h = (s["x"].float() + s["res"].float()).to(dt) if s["residual"] else s["x"]
    x, w = h.float(), s["weight"].float()
    rstd = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    v = x * rstd * w
    out = {"rstd": rstd[:, 0]}
    if s["residual"]:
        out["h"] = h
    if s["out"] == "y":
        out["y"] = v.to(dt)
    else:
        out["q"], out["sf"] = _quantised(v, s["out"])
    if s["grad"]:
        dy = s["dy"].float()
        n, wdy = x * rstd, dy * w
        out["dx"] = (s["dh"].float() + rstd * (wdy - n * (wdy * n).mean(1, keepdim=True))).to(dt)
        out["dw"] = (dy * n).sum(0)
    return out


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z * _sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return z


def _dact_of(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = _sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    p = _sigmoid(c * (z + 0.044715 * z * z * z))
    return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)


def _weight_values(q, s):
    """fp32 values of e4m3 codes [..., N, K] with scales [..., ceil(N / 128), K / 128]."""
    N, K = q.shape[-2:]
    rows = torch.arange(N, device=DEV) // 128
    v = q.view(FP8).float().unflatten(-1, (K // 128, 128))
    return (v * s[..., rows, :, None]).flatten(-2)


def _epilogue(s):
    M, K = s["A"].shape
    a = (s["A"].view(FP8).float().reshape(M, K // 128, 128) * s["sfa"].t()[..., None]).reshape(M, K)
    z = torch.mm(a, _weight_values(s["B"], s["sfb"]).t())
    if s["bias"]:
        z = z + s["b"]
    d = _act(z, s["act"])
    if s["residual"]:
        d = d + s["res"].float()
    out = {"D": d.to(torch.bfloat16)}
    if s["pre"]:
        out["Z"] = z.to(torch.bfloat16)
    return out


def _dact(s):
    dz = s["dy"].float()
    if s["act"] != "none":
        dz = dz * _dact_of(s["Z"].float(), s["act"])
    out = {"dz": dz.to(torch.bfloat16)}
    if s["quant"]:
        out["q"], out["sf"] = _quantised(dz, "fp8")
    if s["bias"]:
        out["db"] = dz.sum(0)
    return out


def _fp4_values(codes, words):
    """fp32 values of packed codes [..., N, K / 2] with scale words [..., K / 128, N]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = _fp4_grid()[(c & 7).long()] * torch.where(c >= 8, -1.0, 1.0)
    e = words.transpose(-1, -2).contiguous().view(torch.uint8).int() - 127
    return torch.ldexp(v.unflatten(-1, (-1, 32)), e[..., None]).flatten(-2)


def _experts(s):
    T, G, H, I = s["T"], s["G"], s["H"], s["I"]
    values = _weight_values if s["fmt"] == "fp8" else _fp4_values
    # every token through every expert; the routing weight of a pair that was not chosen is zero
    gu = torch.mm(s["x"].float(), values(s["w1"], s["s1"]).reshape(G * 2 * I, H).t()).reshape(T, G, 2, I)
    hit = s["idx"][..., None] == s["first"] + torch.arange(G, device=DEV)
    r = (s["w"][..., None] * hit).sum(1)
    h = gu[:, :, 0] * _sigmoid(gu[:, :, 0]) * gu[:, :, 1] * r[..., None]
    w2 = values(s["w2"], s["s2"]).transpose(0, 1).reshape(H, G * I)
    return torch.mm(h.reshape(T, G * I), w2.t()).to(torch.bfloat16)


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def nearest(v):
        """v, up to 448 in magnitude, on the grid of e4m3: multiples of 2^-9 below 2^-6, else of an eighth of v's power of two."""
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0**-9)))
        e = e + (torch.exp2(e + 1) <= v.abs()).to(f64) - (torch.exp2(e) > v.abs().clamp(min=2.0**-9)).to(f64)
        step = torch.exp2(torch.clamp(e, min=-6) - 3)
        return torch.round(v / step) * step

    def quant(v, kind):
        M, K = v.shape
        q, scales = torch.empty_like(v), torch.empty(K // 128, M, dtype=f64, device=DEV)
        for j in range(K // 128):
            b = v[:, 128 * j:128 * j + 128]
            a = b.abs().amax(1) / 448
            a = torch.where(a == 0, 1.0, a)
            if kind == "ue8m0":
                a = torch.exp2(torch.ceil(torch.log2(a)))
            scales[j] = a
            q[:, 128 * j:128 * j + 128] = nearest(b / a[:, None])
        if kind == "fp8":
            return q, scales
        packed = torch.full(((K + 511) // 512, M, 4), 2.0**-127, dtype=f64, device=DEV)
        for j in range(K // 128):
            packed[j // 4, :, j % 4] = scales[j]
        return q, packed.flatten(1)

    if op == "norm":
        h = s["x"] if s["res"] is None else (s["x"].double() + s["res"].double()).to(s["x"].dtype)
        x = h.double().requires_grad_(case["grad"])
        w = s["weight"].double().requires_grad_(case["grad"])
        rstd = torch.rsqrt(x.square().sum(1) / case["K"] + EPS)
        y = w * (x * rstd[:, None])
        out = {"rstd": rstd.detach()}
        if case["residual"]:
            out["h"] = h.double()
        if case["out"] == "y":
            out["y"] = y.detach()
        else:
            out["q"], out["sf"] = quant(y, case["out"])
        if case["grad"]:
            dx, out["dw"] = torch.autograd.grad((y * s["dy"].double()).sum(), (x, w))
            out["dx"] = dx + s["dh"].double()
        return out

    def act(z):
        kind = case["act"]
        if kind == "relu":
            return torch.relu(z)
        if kind == "silu":
            return z * torch.sigmoid(z)
        if kind == "gelu":
            return z * torch.special.ndtr(z)
        if kind == "gelu_tanh":
            return z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3))) / 2
        return z * 1

    if op == "dact":
        dz = s["dy"].double()
        if case["act"] != "none":
            z = s["Z"].double().requires_grad_(True)
            dz = torch.autograd.grad(act(z), z, dz)[0]
        out = {"dz": dz}
        if case["quant"]:
            out["q"], out["sf"] = quant(dz, "fp8")
        if case["bias"]:
            out["db"] = dz.sum(0)
        return out

    def block_weight(q, sc):
        v = q.view(FP8).double()
        for i in range(sc.shape[0]):
            for j in range(sc.shape[1]):
                v[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= sc[i, j].double()
        return v

    def fp4_weight(codes, words):
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=f64, device=DEV)
        v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=f64, device=DEV)
        v[:, 0::2], v[:, 1::2] = table[(codes % 16).long()], table[(codes // 16).long()]
        for b in range(v.shape[1] // 32):
            v[:, 32 * b:32 * b + 32] *= torch.exp2(((words[b // 4].long() >> (8 * (b % 4))) & 255).double() - 127)[:, None]
        return v

    if op == "epilogue":
        a = s["A"].view(FP8).double()
        for j in range(case["K"] // 128):
            a[:, 128 * j:128 * j + 128] *= s["sfa"][j].double()[:, None]
        z = a @ block_weight(s["B"], s["sfb"]).t() + (0 if s["b"] is None else s["b"].double())
        d = act(z) + (0 if s["res"] is None else s["res"].double())
        return {"D": d, "Z": z} if case["pre"] else {"D": d}
    I = case["I"]
    value = block_weight if case["fmt"] == "fp8" else fp4_weight
    y = torch.zeros(case["T"], case["H"], dtype=f64, device=DEV)
    for e in range(case["G"]):
        t, j = torch.nonzero(s["idx"] == case["first"] + e, as_tuple=True)
        if not len(t):
            continue
        gu = s["x"][t].double() @ value(s["w1"][e], s["s1"][e]).t()
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y.index_add_(0, t, s["w"][t, j].double()[:, None] * (h @ value(s["w2"][e], s["s2"][e]).t()))
    return y


# ---- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "norm":
        n, b = case["M"] * case["K"], 2 if case["dtype"] == "bf16" else 4
        t = n * b * (3 if case["residual"] else 1) + case["K"] * b + 4 * case["M"]  # x, residual, their sum; weight; rstd
        t += n * b if case["out"] == "y" else n + n // 128 * (4 if case["out"] == "fp8" else 1)
        # backward: gradients of the output and of the sum, the sum, the gradient; the weight's gradient
        return {"bytes": t + (4 * n * b + 4 * case["K"] if case["grad"] else 0), "flops": 5 * n + (9 * n if case["grad"] else 0)}
    if op == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K + 4 * M * K // 128 + N * K // 4096 + 4 * N * case["bias"] + 2 * M * N * (1 + case["residual"] + case["pre"]),
                "flops": 2 * M * N * K}
    if op == "dact":
        n = case["M"] * case["N"]
        return {"bytes": n * (4 + 2 * (case["act"] != "none")) + (n + n // 32 if case["quant"] else 0) + 4 * case["N"] * case["bias"], "flops": 10 * n}
    T, k, E, G, H, I = (case[n] for n in ("T", "k", "E", "G", "H", "I"))
    live = T * (1 - case["pad"])
    active = G * (1 - (1 - k / E) ** live)  # experts with a token, as expected of even routing
    per = 3 * H * I * (1 + 1 / 4096 if case["fmt"] == "fp8" else 0.5 + 1 / 32)
    return {"bytes": active * per + 4 * T * H + 8 * T * k, "flops": 6 * H * I * live * k * G / E}
