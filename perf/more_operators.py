"""The experts' products that stand around dispatch and combine, as measured cases.

  quant        activation rows or weights -> 8-bit floating-point (e4m3) codes with one scale
               for each block of 1 x 128 or 128 x 128 values
  fp8          product of such codes, dense, grouped over the experts' receive planes, or
               grouped over rows that stand one expert after another
  forward      one linear map per expert over rows that stand one expert after another (bf16)
  input_grad   its gradient with respect to the rows
  weight_grad  its gradient with respect to the maps

`run` computes each in its plain form with elementary torch operations, or, with `own` set,
through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128


def listed():
    return [
        # decode rows ahead of an 8-bit product: 8 ranks x 64 tokens
        {"name": "quant decode", "op": "quant", "rows": 512, "hidden": 7168, "dtype": "bf16",
         "block_rows": 1},
        # prefill rows: 8 ranks x 4096 tokens
        {"name": "quant prefill", "op": "quant", "rows": 32768, "hidden": 7168,
         "dtype": "bf16", "block_rows": 1},
        # a dense projection at decode: the weights' bytes are the floor
        {"name": "fp8 decode", "op": "fp8", "form": "dense", "groups": 1, "rows": 16, "n": 7168,
         "h": 4096},
        # odd sizes: a short chunk of a prompt, no extent a multiple of a tile or a block
        {"name": "fp8 odd", "op": "fp8", "form": "dense", "groups": 1, "rows": 333, "n": 1000,
         "h": 1040},
        # a dense projection at prefill: the multiplications are the floor
        {"name": "fp8 prefill", "op": "fp8", "form": "dense", "groups": 1, "rows": 8192,
         "n": 4096, "h": 7168},
        # the experts' planes after dispatch: ragged counts, some experts without a row
        {"name": "fp8 planes", "op": "fp8", "form": "planes", "groups": 32, "rows": 1024,
         "n": 4096, "h": 2048},
        # one token, sorted by its experts, through a small layer's gate and up maps
        {"name": "forward one token", "op": "forward", "groups": 128, "rows": 8, "n": 1536,
         "h": 2048},
        # a prefill batch sorted by expert: 2048 tokens, 8 experts each
        {"name": "forward prefill", "op": "forward", "groups": 32, "rows": 16384, "n": 4096,
         "h": 2048},
        # a short batch's way back, ragged and odd
        {"name": "input grad odd", "op": "input_grad", "groups": 7, "rows": 999, "n": 1000,
         "h": 1032},
        # the way back of the prefill batch: a training step
        {"name": "input grad step", "op": "input_grad", "groups": 32, "rows": 16384, "n": 4096,
         "h": 2048},
        {"name": "weight grad odd", "op": "weight_grad", "groups": 7, "rows": 999, "n": 1000,
         "h": 1032, "grad": "bf16"},
        {"name": "weight grad step", "op": "weight_grad", "groups": 32, "rows": 16384,
         "n": 4096, "h": 2048, "grad": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["quant", "fp8", "forward", "input_grad", "weight_grad"])
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 16384), "hidden": _mult(rng, 128, 7168, 16),
                "dtype": rng.choice(["bf16", "fp32"]), "block_rows": rng.choice([1, BLOCK])}
    if op == "fp8":
        form = rng.choice(["dense", "planes", "ragged"])
        groups = 1 if form == "dense" else _log(rng, 2, 32)
        n, h = _log(rng, 64, 4096), _mult(rng, 128, 7168, 16)
        most = 8192 // groups if form == "planes" else 8192
        return {"op": op, "form": form, "groups": groups, "rows": min(_log(rng, 1, 8192), most),
                "n": n, "h": h}
    n, h = _mult(rng, 64, 4096, 8), _mult(rng, 64, 7168, 8)
    groups = min(_log(rng, 1, 128), 32 * 4096 * 2048 // (n * h))
    rows = min(_log(rng, 1, 16384), 16384 * 4096 * 2048 // (n * h))
    case = {"op": op, "groups": groups, "rows": rows, "n": n, "h": h}
    if op == "weight_grad":
        case["grad"] = rng.choice(["bf16", "fp32"])
    return case


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 2 + 1)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _codes(shape, g):
    """Codes as a scaling to the largest finite value leaves normal values."""
    c = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, 120.0, generator=g)
    return c.clamp_(-448, 448).to(torch.float8_e4m3fn)


def _scales(shape, mean, g):
    return mean * (0.5 + torch.rand(shape, generator=g, device=DEV))


def _normal(shape, std, g):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def _plane_counts(case, seed):
    """Rows in use of each plane: routed traffic is uneven, and some experts get nothing."""
    g = torch.Generator().manual_seed(seed + 5)
    share = torch.rand(case["groups"], generator=g) ** 2
    c = (share * (case["rows"] + 1)).to(torch.int32).clamp_(0, case["rows"])
    c[int(torch.randint(case["groups"], (1,), generator=g))] = 0
    return c


def _offsets(case, seed):
    """Where each expert's rows begin, and the end of the last one's: every row drew its
    expert, some experts more often than others; in some batches the last rows are padding."""
    g = torch.Generator().manual_seed(seed + 7)
    share = torch.rand(case["groups"], generator=g) ** 2 + 1e-6
    rows = case["rows"] - (seed % 2) * (case["rows"] // 16)
    e = torch.multinomial(share, rows, replacement=True, generator=g)
    c = torch.bincount(e, minlength=case["groups"])
    return torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "quant":
        x = torch.randn((case["rows"], case["hidden"]), generator=g, device=DEV)
        x *= torch.exp(torch.randn((case["rows"], 1), generator=g, device=DEV))
        s["x"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    elif op == "fp8":
        G, M, N, H = case["groups"], case["rows"], case["n"], case["h"]
        lead = () if case["form"] == "ragged" else (G,)
        s["xq"], s["wq"] = _codes((*lead, M, H), g), _codes((G, N, H), g)
        s["sx"] = _scales((*lead, M, _blocks(H)), 1.0 / 120.0, g)
        s["sw"] = _scales((G, _blocks(N), _blocks(H)), 1.0 / (120.0 * math.sqrt(H)), g)
        # the output buffer that the program keeps: rows of no expert stay as they are
        s["out"] = torch.zeros((*lead, M, N), dtype=torch.bfloat16, device=DEV)
        if case["form"] == "planes":
            s["counts"] = _plane_counts(case, seed).to(DEV)
        elif case["form"] == "ragged":
            s["host_offsets"] = _offsets(case, seed)
            s["offsets"] = s["host_offsets"].to(DEV)
    else:
        G, M, N, H = case["groups"], case["rows"], case["n"], case["h"]
        s["host_offsets"] = _offsets(case, seed)
        s["offsets"] = s["host_offsets"].to(DEV)
        if op != "input_grad":
            s["x"] = _normal((M, H), 1.0, g)
        if op != "forward":
            s["dy"] = _normal((M, N), 1.0, g)
        if op != "weight_grad":
            s["w"] = _normal((G, N, H), 1.0 / math.sqrt(H if op == "forward" else N), g)
        shape = {"forward": (M, N), "input_grad": (M, H), "weight_grad": (G, N, H)}[op]
        s["out"] = torch.zeros(shape, device=DEV,
                               dtype=torch.float32 if case.get("grad") == "fp32"
                               else torch.bfloat16)
    if own:
        from combine_topk_ids_rank_gb300 import moe_a2a
        s["api"] = moe_a2a
        if op == "fp8":
            s["handle"] = moe_a2a.MoeGemmFp8(G, M, N, H, DEV)
        elif op != "quant":
            s["handle"] = moe_a2a.MoeGemmRagged(G, M, N, H, DEV)
    return s


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


# ---- the package's entry points ------------------------------------------------

_run_own = {
    "quant": lambda s: s["api"].quantize_blocks_fp8(s["x"], s["case"]["block_rows"]),
    "fp8": lambda s: s["handle"].gemm(s["xq"], s["sx"], s["wq"], s["sw"],
                                      counts=s.get("counts"), offsets=s.get("offsets"),
                                      out=s["out"]),
    "forward": lambda s: s["handle"].forward(s["x"], s["w"], s["offsets"], out=s["out"]),
    "input_grad": lambda s: s["handle"].input_grad(s["dy"], s["w"], s["offsets"], out=s["out"]),
    "weight_grad": lambda s: s["handle"].weight_grad(s["dy"], s["x"], s["offsets"],
                                                     out=s["out"]),
}


# ---- the plain forms -------------------------------------------------------------

def _over_blocks(scale, rows, cols, block_rows):
    """A scale for each block, repeated for each value of it."""
    scale = scale.repeat_interleave(BLOCK, -1)[..., :cols]
    return scale if block_rows == 1 else scale.repeat_interleave(block_rows, -2)[..., :rows, :]


def _plain_quant(s):
    x, b = s["x"].float(), s["case"]["block_rows"]
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % b))
    amax = pad.abs().view(-1, b, _blocks(cols), BLOCK).amax((1, 3))
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    q = x / _over_blocks(scale, rows, cols, b)
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _at(s):
    """The rows of each expert, padded to the longest, and which of them exist."""
    host, off = s["host_offsets"], s["offsets"].long()
    most = max(1, int((host[1:] - host[:-1]).max()))
    at = off[:-1, None] + torch.arange(most, device=DEV)
    return at.clamp(max=s["case"]["rows"] - 1), at < off[1:, None]


def _rows_of(x, at, live):
    return torch.where(live[:, :, None], x[at], torch.zeros((), device=DEV))


def _plain_fp8(s):
    M, N, H = (s["case"][n] for n in ("rows", "n", "h"))
    x = s["xq"].float() * _over_blocks(s["sx"], M, H, 1)
    w = s["wq"].float() * _over_blocks(s["sw"], N, H, BLOCK)
    if s["case"]["form"] == "ragged":
        return _placed(s, w.transpose(1, 2), x)
    y = torch.bmm(x, w.transpose(1, 2)).to(torch.bfloat16)
    if s["case"]["form"] == "planes":
        row = torch.arange(M, device=DEV)
        y = torch.where((row[None] < s["counts"][:, None])[:, :, None], y, s["out"])
    return y


def _placed(s, w, x):
    """Each row through its expert's map; the other rows of `out` stay as they are."""
    at, live = _at(s)
    y = torch.bmm(_rows_of(x, at, live), w)
    s["out"][at[live]] = y[live].to(torch.bfloat16)
    return s["out"]


def _plain_weight_grad(s):
    at, live = _at(s)
    dy, x = _rows_of(s["dy"].float(), at, live), _rows_of(s["x"].float(), at, live)
    return torch.bmm(dy.transpose(1, 2), x).to(s["out"].dtype)


_run_plain = {
    "quant": _plain_quant, "fp8": _plain_fp8,
    "forward": lambda s: _placed(s, s["w"].float().transpose(1, 2), s["x"].float()),
    "input_grad": lambda s: _placed(s, s["w"].float(), s["dy"].float()),
    "weight_grad": _plain_weight_grad,
}


# ---- from the definitions, in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        r, b = case["rows"], case["block_rows"]
        mag = s["x"].double().abs()
        tall = torch.stack([mag[i:i + b].max(0).values for i in range(0, r, b)]) if b > 1 else mag
        amax = torch.stack([tall[:, c:c + BLOCK].max(1).values
                            for c in range(0, case["hidden"], BLOCK)], 1)
        return None, torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    out = s["out"].double()
    for e in range(case["groups"]):
        if "host_offsets" in s:
            lo, hi = int(s["host_offsets"][e]), int(s["host_offsets"][e + 1])
        else:
            lo, hi = 0, int(s["counts"][e]) if "counts" in s else case["rows"]
        if lo == hi:
            continue
        if op == "fp8":
            here = out if case["form"] == "ragged" else out[e]
            x, sx = (s[n] if case["form"] == "ragged" else s[n][e] for n in ("xq", "sx"))
            acc = 0.0
            for b in range(_blocks(case["h"])):
                cols = slice(b * BLOCK, (b + 1) * BLOCK)
                each = s["sw"][e, :, b].double()[torch.arange(case["n"], device=DEV) // BLOCK]
                part = x[lo:hi, cols].double() @ s["wq"][e][:, cols].double().T
                acc = acc + part * sx[lo:hi, b].double()[:, None] * each
            here[lo:hi] = acc
        elif op == "forward":
            out[lo:hi] = s["x"][lo:hi].double() @ s["w"][e].double().T
        elif op == "input_grad":
            out[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
        else:
            out[e] = s["dy"][lo:hi].double().T @ s["x"][lo:hi].double()
    return out


def _used(groups, rows):
    """Experts that at least one row drew, by the mean over the offsets' distribution."""
    n = 256
    share = [((i + 0.5) / n) ** 2 * 3.0 / groups for i in range(n)]
    return groups * sum(1.0 - max(0.0, 1.0 - p) ** rows for p in share) / n


def work(case):
    op = case["op"]
    if op == "quant":
        r, h = case["rows"], case["hidden"]
        scales = (r if case["block_rows"] == 1 else _blocks(r)) * _blocks(h)
        return {"bytes": r * h * (3 if case["dtype"] == "bf16" else 5) + 4 * scales,
                "flops": 3 * r * h}
    G, M, N, H = case["groups"], case["rows"], case["n"], case["h"]
    if op == "fp8":
        rows, used = M, G
        if case["form"] == "planes":
            rows = G * M / 3.0  # mean of the counts' distribution
        elif case["form"] == "ragged":
            used = _used(G, M)
        return {"bytes": used * (N * H + 4 * _blocks(N) * _blocks(H))
                + rows * (H + 4 * _blocks(H) + 2 * N), "flops": 2.0 * rows * N * H}
    if op == "weight_grad":
        size = 4 if case["grad"] == "fp32" else 2
        return {"bytes": G * N * H * size + 2 * M * (N + H), "flops": 2.0 * M * N * H}
    return {"bytes": 2 * _used(G, M) * N * H + 2 * M * (N + H), "flops": 2.0 * M * N * H}
