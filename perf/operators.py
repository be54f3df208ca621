"""Cases of the operators of a mixture-of-experts layer around the grouped products, in the forms a program calls them:

gate     router logits -> top-k experts and weights, per-expert counts, balance loss; with its gradient
layout   chosen experts -> row order of the contiguous and masked grouped products
quant    rows (as they are, or gathered by token) -> microscaled 4-bit floats (e2m1, a power-of-two scale per 32), and back
product  D = A . B^T of microscaled 4-bit operands: dense, contiguous by expert, masked by expert
combine  expert rows -> tokens, weighted by the gate; with its gradient

Each has a plain form in elementary 32-bit torch operations, the framework's own call (``own``), and its definition in 64
bits (``exact``)."""

import math
import random

import torch

own = False
DEV = "cuda"
COEF = 0.01  # weight of the balance loss


def listed():
    return [
        # one decode step of 64 sequences through a 256-expert, top-8 router, bfloat16 logits: latency
        {"name": "gate_decode", "op": "gate", "T": 64, "E": 256, "k": 8, "dtype": "bf16", "renorm": True, "grad": False, "pad": 0.0},
        # a training step's router, forward and backward, fp32 logits, a tenth of the tokens being padding
        {"name": "gate_train", "op": "gate", "T": 32768, "E": 256, "k": 8, "dtype": "f32", "renorm": True, "grad": True, "pad": 0.1},
        # one decode step on a GPU that holds 32 of 256 experts: rows of the masked products
        {"name": "layout_decode", "op": "layout", "T": 256, "k": 8, "E": 256, "first": 64, "G": 32, "max_m": 128},
        # a prefill batch over 64 experts: segments of the contiguous products
        {"name": "layout_prefill", "op": "layout", "T": 16384, "k": 8, "E": 64, "first": 0, "G": 64, "max_m": 0},
        # decode activations gathered into the masked rows as they are quantised
        {"name": "quant_gather", "op": "quant", "T": 256, "R": 2051, "K": 7168, "G": 1, "dtype": "bf16", "gather": True},
        # the weights of 8 experts quantised once (and read back, as a check or a fallback does)
        {"name": "quant_weights", "op": "quant", "T": 4096, "R": 4096, "K": 7168, "G": 8, "dtype": "f32", "gather": False},
        # decode: a small batch against one weight
        {"name": "product_small", "op": "product", "form": "dense", "G": 1, "rows": 64, "max_m": 0, "N": 7168, "K": 2048},
        # a long dense product, an odd number of rows
        {"name": "product_dense", "op": "product", "form": "dense", "G": 1, "rows": 4095, "max_m": 0, "N": 4096, "K": 7168},
        # prefill: 8 experts, tokens spread unevenly, segments padded to 128 rows
        {"name": "product_contiguous", "op": "product", "form": "contiguous", "G": 8, "rows": 16384, "max_m": 0, "N": 4096, "K": 7168},
        # decode: 32 experts with up to 128 tokens each, counts on the device
        {"name": "product_masked", "op": "product", "form": "masked", "G": 32, "rows": 2048, "max_m": 128, "N": 4096, "K": 7168},
        # decode: expert outputs back to 256 tokens
        {"name": "combine_decode", "op": "combine", "T": 256, "k": 8, "N": 7168, "grad": False},
        # training: the same for a batch of tokens, with the gradients of rows and weights
        {"name": "combine_train", "op": "combine", "T": 4096, "k": 8, "N": 7168, "grad": True},
    ]


def _log(rng, lo, hi, step=1):
    """A size, a multiple of `step` from lo * step to hi * step, even over its logarithm (3072 is left out)."""
    n = step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n != 3072 else n + step


def draw(rng):
    op = rng.choice(["gate", "layout", "quant", "product", "product", "combine"])
    if op == "gate":
        E = rng.choice([8, 16, 60, 64, 97, 128, 160, 256, 256, 384, 512])
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 10)), "dtype": rng.choice(["bf16", "f32"]),
                "renorm": rng.random() < 0.6, "grad": rng.random() < 0.6, "pad": rng.choice([0.0, 0.0, 0.1, 0.5])}
    if op == "layout":
        E = rng.choice([8, 16, 60, 64, 128, 256])
        G = rng.choice([E, E, max(1, E // 4), max(1, E // 8)])
        return {"op": op, "T": _log(rng, 1, 16384), "k": rng.randint(1, min(E, 8)), "E": E, "first": rng.randint(0, E - G), "G": G,
                "max_m": rng.choice([0, 0, 32, 100, 256])}
    if op == "quant":
        gather = rng.random() < 0.5
        R = _log(rng, 1, 8192)
        return {"op": op, "T": max(1, R // rng.randint(1, 8)) if gather else R, "R": R, "K": _log(rng, 1, 56, 128), "G": 1 if gather else rng.choice([1, 1, 2, 3]),
                "dtype": rng.choice(["bf16", "f32"]), "gather": gather}
    if op == "product":
        form = rng.choice(["dense", "contiguous", "masked"])
        G = 1 if form == "dense" else rng.choice([2, 4, 7, 8, 16])
        max_m = rng.choice([16, 64, 100, 128, 200, 256]) if form == "masked" else 0
        rows = _log(rng, 1, G * max_m) if form == "masked" else _log(rng, 1, 4096) if form == "dense" else _log(rng, G, 8192)
        return {"op": op, "form": form, "G": G, "rows": rows, "max_m": max_m, "N": _log(rng, 8, 256, 16), "K": _log(rng, 2, 56, 128)}
    return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, 8), "N": _log(rng, 8, 448, 16), "grad": rng.random() < 0.5}


# ---- what a program has in hand


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _fp4_grid():
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)


def _quantised(x):
    """Rows [..., K] of fp32 -> (codes [..., K / 2] uint8, low nibble first; scale codes [..., K / 32] uint8), elementary
    operations: the scale is the smallest power of two not below the block's largest magnitude / 6, 1 for a block of zeros."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    s = torch.where(m <= 0.75, e - 3, e - 2)
    s = torch.where(amax == 0, torch.zeros_like(s), s).clamp(-127, 126)
    y = torch.ldexp(b.abs(), -s[..., None])
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = torch.round(y / step) * step
    code = (torch.bucketize(y, _fp4_grid()) + 8 * torch.signbit(b)).to(torch.uint8).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (s + 127).to(torch.uint8)


def _scale_words(s):
    """Scale codes [..., rows, K / 32] -> words [..., K / 128, rows] int32, the four blocks of 128 in a word's bytes."""
    return s.contiguous().view(torch.int32).transpose(-1, -2).contiguous()


def _values(codes, words):
    """The fp32 values of codes [..., rows, K / 2] and scale words [..., K / 128, rows]."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).int()
    v = _fp4_grid()[(c & 7).long()] * torch.where(c >= 8, -1.0, 1.0)
    s = words.transpose(-1, -2).contiguous().view(torch.uint8).int() - 127
    return torch.ldexp(v.reshape(*v.shape[:-1], -1, 32), s[..., None]).reshape(v.shape)


def _routed(T, k, E, seed):
    """k distinct experts of each of T tokens, some experts more popular than others."""
    g = _gen(seed)
    pop = 0.7 * torch.randn(E, device=DEV, generator=g)
    return torch.topk(pop + torch.randn(T, E, device=DEV, generator=g), k, dim=1).indices.int().contiguous()


def _activations(shape, seed):
    g = _gen(seed)
    x = torch.randn(shape, device=DEV, generator=g)
    return torch.where(torch.rand(shape, device=DEV, generator=g) < 1e-3, 20 * x, x)


def prepare(case, seed):
    def expert_rows(total, G, most, seed):
        """Rows of each of G experts, uneven, `total` in all and at most `most` each."""
        r = random.Random(seed)
        share = [r.random() + 0.05 for _ in range(G)]
        n = [min(most, int(total * s / sum(share))) for s in share]
        left = total - sum(n)
        for i in list(range(G)) * 2:
            more = min(left, most - n[i])
            n[i], left = n[i] + more, left - more
        return n

    op = case["op"]
    s = dict(case)
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        g = _gen(seed)
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = (1.5 * torch.randn(T, E, device=DEV, generator=g) + 0.7 * torch.randn(E, device=DEV, generator=g)).to(dt)
        s["valid"] = torch.rand(T, device=DEV, generator=g) >= case["pad"] if case["pad"] else None
        s["dw"] = torch.randn(T, k, device=DEV, generator=g)
        s["dloss"] = torch.ones(1, device=DEV)
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(T, k, device=DEV)
        s["counts"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["prob_sum"] = torch.empty(E, device=DEV)
        s["loss"] = torch.empty(1, device=DEV)
        s["dlogits"] = torch.empty_like(s["logits"])
        s["ws"] = torch.zeros(4 << 20, dtype=torch.uint8, device=DEV)
    elif op == "layout":
        T, k, G, max_m = case["T"], case["k"], case["G"], case["max_m"]
        s["idx"] = _routed(T, k, case["E"], seed)
        rows = G * max_m if max_m else (T * k + 127 * G + 127) // 128 * 128
        s["counts"] = torch.empty(G, dtype=torch.int32, device=DEV)
        s["m_indices"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["row_token"] = torch.empty((G, max_m) if max_m else (rows,), dtype=torch.int32, device=DEV)
        s["row_of"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["ws"] = torch.zeros(4 << 20, dtype=torch.uint8, device=DEV)
    elif op == "quant":
        T, R, K, G = case["T"], case["R"], case["K"], case["G"]
        lead = (G,) if G > 1 else ()
        s["x"] = _activations(lead + (T, K), seed).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["rows"] = None
        if case["gather"]:  # a quarter of the rows hold no token
            rows = torch.randint(0, T, (R,), device=DEV, generator=_gen(seed + 1), dtype=torch.int32)
            s["rows"] = torch.where(torch.rand(R, device=DEV, generator=_gen(seed + 2)) < 0.25, -1, rows).int()
        s["q"] = torch.zeros(lead + (R, K // 2), dtype=torch.uint8, device=DEV)
        s["sf"] = torch.zeros(lead + (K // 128, R), dtype=torch.int32, device=DEV)
        s["y"] = torch.empty(lead + (R, K), dtype=torch.bfloat16, device=DEV)
    elif op == "product":
        G, rows, N, K, max_m, form = (case[n] for n in ("G", "rows", "N", "K", "max_m", "form"))
        lead = (G,) if form != "dense" else ()
        q, e = _quantised(torch.randn(lead + (N, K), device=DEV, generator=_gen(seed + 1)) / math.sqrt(K))
        s["B"], s["sfb"] = q, _scale_words(e)
        if form == "contiguous":
            counts = expert_rows(rows, G, rows, seed)
            M = (rows + 127 * G + 127) // 128 * 128
            expert, start = torch.full((M,), -1, dtype=torch.int32), 0
            for e_, n in enumerate(counts):
                expert[start:start + n] = e_
                start += (n + 127) // 128 * 128
            s["m_indices"], s["most"] = expert.to(DEV), max(counts)
        elif form == "masked":
            M = G * max_m
            s["masked_m"] = torch.tensor(expert_rows(rows, G, max_m, seed), dtype=torch.int32, device=DEV)
        else:
            M = rows
        q, e = _quantised(_activations((M, K), seed))
        if form == "masked":
            q, e = q.reshape(G, max_m, -1), e.reshape(G, max_m, -1)
        s["A"], s["sfa"] = q, _scale_words(e)
        s["D"] = torch.zeros(q.shape[:-1] + (N,), dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV) if form == "dense" else None
    else:
        T, k, N = case["T"], case["k"], case["N"]
        g = _gen(seed)
        R = (T * k * 5 // 4 + 127) // 128 * 128  # padded segments
        s["rows"] = torch.randn(R, N, device=DEV, generator=g).to(torch.bfloat16)
        row_of = torch.randperm(R, device=DEV, generator=g)[: T * k].reshape(T, k)
        s["row_of"] = torch.where(torch.rand(T, k, device=DEV, generator=g) < 0.02, -1, row_of).int()  # choices past a capacity
        s["w"] = torch.softmax(torch.randn(T, k, device=DEV, generator=g), -1)
        s["dy"] = torch.randn(T, N, device=DEV, generator=g).to(torch.bfloat16)
        s["y"] = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        s["drows"] = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
        s["dw"] = torch.empty(T, k, device=DEV)
    return s


# ---- one pass


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from moe_grouped_matmul_amd import dg

    op = s["op"]
    if op == "gate":
        dg.dg_moe_gate(s["logits"], s["idx"], s["w"], s["counts"], s["prob_sum"], s["loss"], renorm=s["renorm"], loss_coef=COEF,
                       valid=s["valid"], workspace=s["ws"])
        out = {"idx": s["idx"], "w": s["w"], "counts": s["counts"], "prob_sum": s["prob_sum"], "loss": s["loss"]}
        if s["grad"]:
            dg.dg_moe_gate_bwd(s["logits"], s["idx"], s["w"], s["counts"], s["dw"], s["dloss"], s["dlogits"], renorm=s["renorm"],
                               loss_coef=COEF)
            out["dlogits"] = s["dlogits"]
        return out
    if op == "layout":
        if s["max_m"]:
            dg.dg_moe_layout_masked(s["idx"], s["counts"], s["row_token"], s["row_of"], first_expert=s["first"], workspace=s["ws"])
            return {"counts": s["counts"], "row_token": s["row_token"], "row_of": s["row_of"]}
        dg.dg_moe_layout_contiguous(s["idx"], s["counts"], s["m_indices"], s["row_token"], s["row_of"], first_expert=s["first"],
                                    workspace=s["ws"])
        return {"counts": s["counts"], "m_indices": s["m_indices"], "row_token": s["row_token"], "row_of": s["row_of"]}
    if op == "quant":
        dg.dg_quant_mxfp4(s["x"], s["q"], s["sf"], row_token=s["rows"])
        dg.dg_dequant_mxfp4(s["q"], s["sf"], s["y"])
        return s["y"]
    if op == "product":
        if s["form"] == "dense":
            dg.dg_mxfp4_gemm_nt(s["A"], s["sfa"], s["B"], s["sfb"], s["D"], workspace=s["ws"])
        elif s["form"] == "contiguous":
            dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(s["A"], s["sfa"], s["B"], s["sfb"], s["D"], s["m_indices"])
        else:
            dg.dg_m_grouped_mxfp4_gemm_nt_masked(s["A"], s["sfa"], s["B"], s["sfb"], s["D"], s["masked_m"])
        return s["D"]
    dg.dg_moe_combine(s["rows"], s["row_of"], s["w"], s["y"])
    if not s["grad"]:
        return {"y": s["y"]}
    dg.dg_moe_combine_bwd(s["dy"], s["rows"], s["row_of"], s["w"], s["drows"], s["dw"])
    return {"y": s["y"], "drows": s["drows"], "dw": s["dw"]}


def _run_plain(s):
    return {"gate": _gate, "layout": _layout, "quant": _quant, "product": _product, "combine": _combine}[s["op"]](s)


def _gate(s):
    x, E, k = s["logits"].float(), s["E"], s["k"]
    valid = s["valid"] if s["valid"] is not None else torch.ones(s["T"], dtype=torch.bool, device=DEV)
    e = torch.exp(x - x.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True) * valid[:, None]
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]  # ties: the lowest expert first
    top = p.gather(1, idx)
    total = top.sum(1, keepdim=True)
    w = top / torch.where(total > 0, total, 1.0) if s["renorm"] else top
    hit = torch.zeros_like(p).scatter_(1, idx, 1.0) * valid[:, None]
    counts = hit.sum(0)
    n, pairs = valid.sum().float(), counts.sum()
    prob_sum = p.sum(0)
    scale = COEF * E / (pairs.clamp(min=1) * n.clamp(min=1))
    loss = scale * (counts * prob_sum).sum()
    out = {"idx": torch.where(valid[:, None], idx, -1).int(), "w": w, "counts": torch.cat((counts, n[None])).int(),
           "prob_sum": prob_sum, "loss": loss[None]}
    if s["grad"]:
        dw = s["dw"]
        dtop = (dw - (dw * w).sum(1, keepdim=True)) / torch.where(total > 0, total, 1.0) if s["renorm"] else dw
        dp = torch.zeros_like(p).scatter_(1, idx, dtop) + s["dloss"] * scale * counts
        out["dlogits"] = (p * (dp - (dp * p).sum(1, keepdim=True))).to(s["logits"].dtype)
    return out


def _layout(s):
    T, k, G, max_m = s["T"], s["k"], s["G"], s["max_m"]
    e = s["idx"].reshape(-1).long() - s["first"]
    here = (e >= 0) & (e < G)
    e = torch.where(here, e, G)
    order = torch.sort(e, stable=True).indices
    counts = (e[:, None] == torch.arange(G, device=DEV)).sum(0)
    held = counts.clamp(max=max_m) if max_m else counts
    start = torch.arange(G, device=DEV) * max_m if max_m else torch.cumsum((counts + 127) // 128 * 128, 0) - (counts + 127) // 128 * 128
    first = torch.cat((torch.cumsum(counts, 0) - counts, torch.zeros(1, dtype=torch.long, device=DEV)))
    rank = torch.empty_like(e)
    rank[order] = torch.arange(T * k, device=DEV) - first[e[order]]
    kept = here & (rank < max_m) if max_m else here
    row = torch.where(kept, torch.cat((start, start[:1]))[e] + rank, -1)
    rows = s["row_token"].numel()
    # rows that hold nothing go to one place past the end
    at = torch.where(kept, row, rows)
    row_token = torch.full((rows + 1,), -1, dtype=torch.long, device=DEV).scatter_(0, at, torch.arange(T * k, device=DEV) // k)[:rows]
    out = {"counts": held.int(), "row_token": row_token.int().reshape(s["row_token"].shape), "row_of": row.int().reshape(T, k)}
    if not max_m:
        out["m_indices"] = torch.full((rows + 1,), -1, dtype=torch.long, device=DEV).scatter_(0, at, e)[:rows].int()
    return out


def _quant(s):
    x = s["x"].float()
    if s["rows"] is not None:
        x = torch.where(s["rows"][:, None] >= 0, x[s["rows"].clamp(min=0).long()], 0.0)
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    scale = torch.where(m <= 0.75, e - 3, e - 2).clamp(-127, 126)
    y = torch.ldexp(b.abs(), -scale)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return torch.copysign(torch.ldexp(torch.round(y / step) * step, scale), b).reshape(x.shape).to(torch.bfloat16)


def _product(s):
    a, b = _values(s["A"], s["sfa"]), _values(s["B"], s["sfb"])
    if s["form"] == "dense":
        return torch.mm(a, b.t()).to(torch.bfloat16)
    bt = b.transpose(1, 2).contiguous()
    if s["form"] == "masked":
        there = torch.arange(s["max_m"], device=DEV) < s["masked_m"][:, None]
        return torch.where(there[..., None], torch.bmm(a, bt), 0.0).to(torch.bfloat16)
    # the experts' rows side by side, as many places each as the fullest has rows
    e = s["m_indices"].long()
    G, cap, M = s["G"], s["most"], e.numel()
    hot = e[:, None] == torch.arange(G, device=DEV)
    rank = (torch.cumsum(hot, 0) - 1).gather(1, e.clamp(min=0)[:, None])[:, 0]
    place = torch.where(e >= 0, e * cap + rank, G * cap)
    row = torch.full((G * cap + 1,), M, device=DEV).scatter_(0, place, torch.arange(M, device=DEV))[: G * cap]
    d = torch.bmm(torch.cat((a, a.new_zeros(1, a.shape[1])))[row].reshape(G, cap, -1), bt).reshape(G * cap, -1)
    return torch.cat((d, d.new_zeros(1, d.shape[1])))[place].to(torch.bfloat16)


def _combine(s):
    row, w = s["row_of"].long(), s["w"]
    there = row >= 0
    x = torch.where(there[..., None], s["rows"].float()[row.clamp(min=0)], 0.0)
    out = {"y": (w[..., None] * x).sum(1).to(torch.bfloat16)}
    if s["grad"]:
        dy = s["dy"].float()
        R = s["rows"].shape[0]
        d = torch.zeros(R + 1, s["N"], device=DEV)
        d[torch.where(there, row, R).reshape(-1)] = (w[..., None] * dy[:, None]).reshape(-1, s["N"])
        out["drows"] = d[:R].to(torch.bfloat16)
        out["dw"] = (x * dy[:, None]).sum(2)
    return out


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "layout":
        return None  # whole numbers only
    if op == "gate":
        x = s["logits"].double()
        T, E, k = case["T"], case["E"], case["k"]
        live = torch.ones(T, 1, dtype=torch.float64, device=DEV) if s["valid"] is None else s["valid"].double()[:, None]
        x.requires_grad_(True)
        p = torch.softmax(x, 1)
        # an expert is chosen where fewer than k others are above it, a lower one being above its equals
        key = torch.arange(E, device=DEV)
        rank = torch.zeros(T, E, dtype=torch.int64, device=DEV)
        for j in range(E):
            c = x.detach()[:, j:j + 1]
            rank += (c > x.detach()) | ((c == x.detach()) & (j < key))
        place = torch.argsort(rank, dim=1)[:, :k]
        top = torch.gather(p, 1, place)
        w = (top / top.sum(1, keepdim=True) if case["renorm"] else top) * live
        counts = ((rank < k).double() * live).sum(0)
        n = live.sum()
        prob_sum = (p * live).sum(0)
        loss = COEF * E * (counts / counts.sum().clamp(min=1) * prob_sum / n.clamp(min=1)).sum()
        out = {"idx": None, "w": w.detach(), "counts": None, "prob_sum": prob_sum.detach(), "loss": loss.detach()[None]}
        if case["grad"]:
            out["dlogits"] = torch.autograd.grad((w * s["dw"].double()).sum() + loss, x)[0]
        return out
    if op == "quant":
        x = s["x"].double()
        if s["rows"] is not None:
            x = torch.cat((x, x.new_zeros(1, x.shape[1])))[s["rows"].long()]  # -1 is the row of zeros
        b = x.unflatten(-1, (-1, 32))
        top = b.abs().amax(-1, keepdim=True)
        ex = torch.ceil(torch.log2(torch.where(top > 0, top, 6.0) / 6))
        ex = ex + (6 * torch.exp2(ex) < top).double() - (6 * torch.exp2(ex - 1) >= top).double() * (top > 0)
        ex = ex.clamp(-127, 126)
        v = b / torch.exp2(ex)
        # the nearest of the sixteen values, of two equally near ones the one with an even mantissa
        grid = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=DEV)  # even ones first
        best, off = torch.zeros_like(v), v.abs()
        for g in grid[1:]:
            d = (v.abs() - g).abs()
            best, off = torch.where(d < off, g, best), torch.minimum(d, off)
        return (torch.sign(v) * best * torch.exp2(ex)).flatten(-2)

    def value(codes, words):
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)
        rows = codes.shape[-2]
        v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=DEV)
        v[..., 0::2], v[..., 1::2] = table[(codes % 16).long()], table[(codes // 16).long()]
        for blk in range(words.shape[-2] * 4):
            sc = (words[..., blk // 4, :].long() >> (8 * (blk % 4))) & 255
            v[..., 32 * blk:32 * blk + 32] *= torch.exp2(sc.double() - 127).reshape(*words.shape[:-2], rows, 1)
        return v

    if op == "product":
        G = case["G"]
        if case["form"] == "dense":
            return value(s["A"], s["sfa"]) @ value(s["B"], s["sfb"]).t()
        a = value(s["A"], s["sfa"])
        d = torch.zeros(s["D"].shape, dtype=torch.float64, device=DEV)
        for g in range(G):
            b = value(s["B"][g], s["sfb"][g])
            if case["form"] == "masked":
                n = int(s["masked_m"][g])
                d[g, :n] = a[g, :n] @ b.t()
            else:
                at = torch.nonzero(s["m_indices"] == g)[:, 0]
                d[at] = a[at] @ b.t()
        return d
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device=DEV)
    drows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros(case["T"], case["k"], dtype=torch.float64, device=DEV)
    rows, dy = s["rows"].double(), s["dy"].double()
    for j in range(case["k"]):
        t = torch.nonzero(s["row_of"][:, j] >= 0)[:, 0]
        r = s["row_of"][t, j].long()
        y[t] += s["w"][t, j].double()[:, None] * rows[r]
        drows[r] = s["w"][t, j].double()[:, None] * dy[t]
        dw[t, j] = (rows[r] * dy[t]).sum(1)
    return {"y": y, "drows": drows, "dw": dw} if case["grad"] else {"y": y}


# ---- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        b = 2 if case["dtype"] == "bf16" else 4
        t = T * E * b + T * k * 8 + 8 * E  # logits read, experts and weights written, the sums
        f = 4 * T * E  # exp, sum, probability, its sum over the tokens
        return {"bytes": t + (T * E * b + T * k * 4 if case["grad"] else 0), "flops": f + (4 * T * E if case["grad"] else 0)}
    if op == "layout":
        rows = case["G"] * case["max_m"] if case["max_m"] else (case["T"] * case["k"] + 127 * case["G"] + 127) // 128 * 128
        return {"bytes": 8 * case["T"] * case["k"] + rows * (4 if case["max_m"] else 8) + 4 * case["G"], "flops": 2 * case["T"] * case["k"]}
    if op == "quant":
        b = 2 if case["dtype"] == "bf16" else 4
        live = 0.75 if case["gather"] else 1.0  # rows that hold a token
        n = case["G"] * case["R"] * case["K"]
        packed = n / 2 + n / 32
        return {"bytes": case["G"] * case["T"] * case["K"] * b + live * packed + packed + 2 * n, "flops": 4 * n}
    if op == "product":
        G, N, K, rows = (case[n] for n in ("G", "N", "K", "rows"))
        return {"bytes": (G * N + rows) * (K / 2 + K / 32) + 2 * rows * N, "flops": 2 * rows * N * K}
    n = case["T"] * case["k"] * case["N"]
    fwd = 2 * n + 2 * case["T"] * case["N"] + 8 * case["T"] * case["k"]
    bwd = 2 * case["T"] * case["N"] + 2 * n + 4 * case["T"] * case["k"]  # the gradient read, a row's gradient each, the weights'
    return {"bytes": fwd + (bwd if case["grad"] else 0), "flops": 2 * n + (3 * n if case["grad"] else 0)}
