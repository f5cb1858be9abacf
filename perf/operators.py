"""The language-model operators that stand around dispatch and combine, as measured cases.

  gate    router logits -> the top-k expert ids and weights that dispatch takes
  quant   activation rows -> 8-bit integer codes and one scale per row
  gemm    product of 8-bit integer codes with one scale per token and per output channel,
          dense or grouped over the experts' receive planes
  layer   a whole mixture-of-experts layer (gate and up product, SiLU, down product, gated
          sum) for a few tokens

`run` computes each in its plain form with elementary torch operations, or, with `own` set,
through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, FP8, INT8 = "bf16", "e4m3", "int8"


def listed():
    return [
        # the router of one small decode step: latency is what counts
        {"name": "gate decode", "op": "gate", "tokens": 8, "experts": 256, "k": 8,
         "dtype": "fp32", "scoring": "softmax", "masked": 0},
        # the router of a prefill batch: 8 ranks x 4096 tokens, bf16 logits full of ties
        {"name": "gate prefill", "op": "gate", "tokens": 32768, "experts": 256, "k": 8,
         "dtype": "bf16", "scoring": "sigmoid", "masked": 0},
        # decode rows ahead of an 8-bit product: 8 ranks x 64 tokens
        {"name": "quant decode", "op": "quant", "rows": 512, "hidden": 7168, "dtype": "bf16"},
        # prefill rows: 8 ranks x 4096 tokens
        {"name": "quant prefill", "op": "quant", "rows": 32768, "hidden": 7168,
         "dtype": "bf16"},
        # a dense projection at decode: the weights' bytes are the floor
        {"name": "gemm decode", "op": "gemm", "groups": 1, "rows": 16, "n": 7168, "h": 4096,
         "ragged": 0},
        # odd sizes: a short chunk of a prompt, no extent a multiple of a tile
        {"name": "gemm odd", "op": "gemm", "groups": 1, "rows": 333, "n": 1000, "h": 1040,
         "ragged": 0},
        # a dense projection at prefill: the multiplications are the floor
        {"name": "gemm prefill", "op": "gemm", "groups": 1, "rows": 8192, "n": 4096,
         "h": 7168, "ragged": 0},
        # the experts' planes after dispatch: ragged counts, some experts without a row
        {"name": "gemm planes", "op": "gemm", "groups": 32, "rows": 1024, "n": 4096,
         "h": 2048, "ragged": 1},
        # one token through a small layer: the shortest decode step
        {"name": "layer one token", "op": "layer", "tokens": 1, "hidden": 2048, "inter": 768,
         "experts": 128, "k": 8, "format": BF16, "absent": 0},
        # a decode batch padded to a graph's size: absent tokens, 8-bit float weights,
        # extents that are no multiple of a tile
        {"name": "layer odd e4m3", "op": "layer", "tokens": 5, "hidden": 1424, "inter": 720,
         "experts": 24, "k": 4, "format": FP8, "absent": 2},
        # a wide layer with 8-bit integer weights, 8 sequences at once
        {"name": "layer wide int8", "op": "layer", "tokens": 8, "hidden": 7168, "inter": 2048,
         "experts": 64, "k": 8, "format": INT8, "absent": 0},
        # the largest batch the layer takes: nearly every expert is used
        {"name": "layer batch", "op": "layer", "tokens": 64, "hidden": 2048, "inter": 1024,
         "experts": 64, "k": 8, "format": BF16, "absent": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["gate", "quant", "gemm", "layer"])
    if op == "gate":
        experts = _log(rng, 8, 512)
        return {"op": op, "tokens": min(_log(rng, 1, 32768), 32768 * 256 // experts),
                "experts": experts, "k": rng.randint(1, min(8, experts)),
                "dtype": rng.choice(["fp32", "bf16"]),
                "scoring": rng.choice(["softmax", "sigmoid"]), "masked": rng.randint(0, 1)}
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 16384), "hidden": _mult(rng, 128, 7168, 16),
                "dtype": rng.choice(["bf16", "fp32"])}
    if op == "gemm":
        groups = rng.choice([1, 1, _log(rng, 2, 32)])
        n, h = _log(rng, 64, 4096), _mult(rng, 128, 7168, 16)
        rows = max(1, min(_log(rng, 1, 8192), 8192 // groups))
        return {"op": op, "groups": groups, "rows": rows, "n": n, "h": h,
                "ragged": int(groups > 1)}
    experts = _log(rng, 8, 128)
    k = rng.randint(1, 8)
    hidden, inter = _mult(rng, 256, 7168, 16), _mult(rng, 128, 2048, 16)
    # the plain form holds each (token, expert) pair's weights in 32 bits
    tokens = max(1, min(_log(rng, 1, 64), 64 * 7168 * 2048 // (k * hidden * inter)))
    return {"op": op, "tokens": tokens, "hidden": hidden, "inter": inter, "experts": experts,
            "k": k, "format": rng.choice([BF16, FP8, INT8]),
            "absent": rng.randint(0, tokens // 2)}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 2 + 1)


def _codes(shape, g):
    """Codes as a symmetric 8-bit quantisation of normal values leaves them."""
    c = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, 36.0, generator=g)
    return c.round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, mean, g):
    return mean * (0.5 + torch.rand(shape, generator=g, device=DEV))


def _weights(shape, fmt, g):
    """A stack of linear maps [experts, out, in] and, for 8-bit codes, its channel scales."""
    std = 1.0 / math.sqrt(shape[-1])
    if fmt == BF16:
        return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std,
                                                                            generator=g), None
    if fmt == INT8:
        return _codes(shape, g), _scales(shape[:-1], std / 36.0, g)
    w = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, 100.0, generator=g)
    return (w.clamp_(-448, 448).to(torch.float8_e4m3fn),
            _scales(shape[:-1], std / 100.0, g))


def _counts(case, seed):
    """Rows of each group: routed traffic is uneven, and some experts get nothing."""
    g = torch.Generator().manual_seed(seed + 5)
    share = torch.rand(case["groups"], generator=g) ** 2
    c = (share * (case["rows"] + 1)).to(torch.int32).clamp_(0, case["rows"])
    c[int(torch.randint(case["groups"], (1,), generator=g))] = 0
    return c


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "gate":
        t, e = case["tokens"], case["experts"]
        logits = torch.randn((t, e), generator=g, device=DEV) * 1.5
        if case["masked"]:  # experts that are closed to a token
            logits.masked_fill_(torch.rand((t, e), generator=g, device=DEV) < 0.3, -math.inf)
        s["logits"] = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    elif op == "quant":
        x = torch.randn((case["rows"], case["hidden"]), generator=g, device=DEV)
        x *= torch.exp(torch.randn((case["rows"], 1), generator=g, device=DEV))
        s["x"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    elif op == "gemm":
        G, M, N, H = case["groups"], case["rows"], case["n"], case["h"]
        s["xq"], s["wq"] = _codes((G, M, H), g), _codes((G, N, H), g)
        s["sx"] = _scales((G, M), 1.0 / 36.0, g)
        s["sw"] = _scales((G, N), 1.0 / (36.0 * math.sqrt(H)), g)
        s["counts"] = _counts(case, seed).to(DEV) if case["ragged"] else None
        # the output buffer that the program keeps: rows past a count stay as they are
        s["out"] = torch.zeros((G, M, N), dtype=torch.bfloat16, device=DEV)
    else:
        T, H, I, E, K = (case[n] for n in ("tokens", "hidden", "inter", "experts", "k"))
        s["x"] = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
        logits = torch.randn((T, E), generator=g, device=DEV)
        top = torch.topk(logits, K, dim=-1)
        s["ids"] = top.indices.to(torch.int32)
        s["w"] = torch.softmax(top.values, dim=-1)
        if case["absent"]:
            s["ids"][T - case["absent"]:] = -1
        s["w13"], s["s13"] = _weights((E, 2 * I, H), case["format"], g)
        s["w2"], s["s2"] = _weights((E, H, I), case["format"], g)
    if own:
        from combine_topk_ids_rank_gb300 import moe_a2a
        s["api"] = moe_a2a
        if op == "gate":
            s["scoring"] = {"softmax": moe_a2a.MOE_SCORE_SOFTMAX,
                            "sigmoid": moe_a2a.MOE_SCORE_SIGMOID}[case["scoring"]]
        elif op == "gemm":
            s["handle"] = moe_a2a.MoeGemmInt8(G, M, N, H, DEV)
        elif op == "layer":
            fmt = {BF16: moe_a2a.MOE_FORMAT_BF16, FP8: moe_a2a.MOE_FORMAT_FP8_E4M3,
                   INT8: moe_a2a.MOE_FORMAT_INT8}[case["format"]]
            s["handle"] = moe_a2a.MoeLayerSmall(E, H, I, K, T, fmt, DEV)
    return s


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


# ---- the package's entry points ------------------------------------------------

_run_own = {
    "gate": lambda s: s["api"].topk_gate(s["logits"], s["case"]["k"], s["scoring"]),
    "quant": lambda s: s["api"].quantize_rows_int8(s["x"]),
    "gemm": lambda s: s["handle"].gemm(s["xq"], s["sx"], s["wq"], s["sw"],
                                       counts=s["counts"], out=s["out"]),
    "layer": lambda s: s["handle"].forward(s["x"], s["ids"], s["w"], s["w13"], s["w2"],
                                           w13_scale=s["s13"], w2_scale=s["s2"]),
}


# ---- the plain forms -------------------------------------------------------------

def _plain_gate(s):
    k = s["case"]["k"]
    l = s["logits"].float()
    v, i = torch.sort(l, dim=-1, descending=True, stable=True)  # equal logits: lowest id
    v, i = v[:, :k], i[:, :k]
    if s["case"]["scoring"] == "softmax":
        top = torch.where(torch.isinf(v[:, :1]), torch.zeros_like(v[:, :1]), v[:, :1])
        w = torch.exp(v - top) / torch.exp(l - top).sum(-1, keepdim=True).clamp(min=1e-30)
    else:
        w = 1.0 / (1.0 + torch.exp(-v))
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return torch.where(torch.isinf(v), -1, i).to(torch.int32), w


def _plain_quant(s):
    x = s["x"].float()
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 127.0), torch.ones_like(amax))
    return torch.round(x / scale[:, None]).to(torch.int8), scale


def _plain_gemm(s):
    y = torch.bmm(s["xq"].float(), s["wq"].float().transpose(1, 2))  # sums stay below 2^24
    y = (y * s["sx"][:, :, None] * s["sw"][:, None, :]).to(torch.bfloat16)
    if s["counts"] is not None:
        row = torch.arange(y.shape[1], device=DEV)
        y = torch.where((row[None] < s["counts"][:, None])[:, :, None], y, s["out"])
    return y


def _rows_f32(w, e, scale):
    """The maps of the experts `e` in 32 bits, without their channel scales."""
    if scale is None:
        return w[e].float()
    return w.view(torch.int8)[e].view(w.dtype).float()


def _plain_layer(s):
    T, K = s["ids"].shape
    e = s["ids"].clamp(min=0).long().reshape(-1)
    x = s["x"].float().repeat_interleave(K, 0)
    h = torch.bmm(_rows_f32(s["w13"], e, s["s13"]), x[:, :, None])[:, :, 0]
    if s["s13"] is not None:
        h = h * s["s13"][e]
    gate, up = h.chunk(2, -1)
    act = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.bmm(_rows_f32(s["w2"], e, s["s2"]), act[:, :, None])[:, :, 0]
    if s["s2"] is not None:
        y = y * s["s2"][e]
    w = torch.where(s["ids"] >= 0, s["w"], torch.zeros_like(s["w"]))
    return (y.view(T, K, -1) * w[:, :, None]).sum(1).to(torch.bfloat16)


_run_plain = {"gate": _plain_gate, "quant": _plain_quant, "gemm": _plain_gemm,
              "layer": _plain_layer}


# ---- from the definitions, in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        l = s["logits"].double()
        if case["scoring"] == "softmax":
            score = torch.nan_to_num(torch.softmax(l, -1), nan=0.0)
        else:
            score = torch.sigmoid(l)
        # descending by logit, ascending by id among equals
        order = torch.argsort(-l, dim=-1, stable=True)[:, :case["k"]]
        w = score.gather(1, order)
        total = w.sum(-1, keepdim=True)
        return None, torch.where(total > 0, w / total, torch.zeros_like(w))
    if op == "quant":
        amax = s["x"].double().abs().max(-1).values
        return None, torch.where(amax > 0, amax / 127.0, torch.ones_like(amax))
    if op == "gemm":
        counts = s["counts"].tolist() if case["ragged"] else [case["rows"]] * case["groups"]
        out = s["out"].double()
        for g, c in enumerate(counts):
            if c:
                dot = s["xq"][g, :c].double() @ s["wq"][g].double().T
                out[g, :c] = dot * torch.outer(s["sx"][g, :c].double(), s["sw"][g].double())
        return out
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    ids = s["ids"].tolist()
    for e in sorted({i for row in ids for i in row if i >= 0}):
        toks = [t for t, row in enumerate(ids) if e in row]
        at = [ids[t].index(e) for t in toks]
        a, b = s["w13"][e].double(), s["w2"][e].double()
        if s["s13"] is not None:
            a, b = a * s["s13"][e].double()[:, None], b * s["s2"][e].double()[:, None]
        h = s["x"][toks].double() @ a.T
        gate, up = h[:, :case["inter"]], h[:, case["inter"]:]
        y = (gate * torch.sigmoid(gate) * up) @ b.T
        out[toks] += y * s["w"][toks, at].double()[:, None]
    return out


def work(case):
    op = case["op"]
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": t * (e * (2 if case["dtype"] == "bf16" else 4) + 8 * k),
                "flops": 4 * t * e}
    if op == "quant":
        n = case["rows"] * case["hidden"]
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + 4 * case["rows"],
                "flops": 3 * n}
    if op == "gemm":
        G, M, N, H = case["groups"], case["rows"], case["n"], case["h"]
        share = 1.0 / 3.0 if case["ragged"] else 1.0  # mean of the counts' distribution
        return {"bytes": G * N * (H + 4) + share * G * M * (H + 4 + 2 * N),
                "flops": 2.0 * share * G * M * N * H}
    T, H, I, E, K = (case[n] for n in ("tokens", "hidden", "inter", "experts", "k"))
    live = T - case["absent"]
    used = E * (1.0 - (1.0 - K / E) ** live)  # experts that at least one token names
    size = 2 if case["format"] == BF16 else 1
    scales = 0 if case["format"] == BF16 else 4 * (2 * I + H)
    return {"bytes": used * (3 * H * I * size + scales) + 4 * T * H + 8 * T * K,
            "flops": 6.0 * live * K * H * I}
