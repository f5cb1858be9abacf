"""The layer for a few tokens where its rings are short and turn often (one expert
takes most tokens, tens of units a CTA), against 64 bits.

Tolerance, counted from roundings: n products summed in fp32 by the tensor cores
are off by at most n * 2^-23 of the sum of their magnitudes.  The activations are
carried in two bf16 terms, each off by at most 2^-8 of what it stands for: 2^-16
together.  SiLU in fp32 takes five operations and an exponential of 2 ulp: 2^-20.
The gated sum has a multiply-add per expert, the output one narrowing to bf16, 2^-8.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"
FORMATS = ["bf16", "e4m3", "int8"]


@pytest.fixture(scope="module")
def api():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def weights(E, O, H, fmt, seed):
    g = gen(seed)
    if fmt == "bf16":
        return (torch.randn((E, O, H), generator=g, device=DEV) / H ** 0.5).to(torch.bfloat16), None
    s = (torch.rand((E, O), generator=g, device=DEV) + 0.5) / H ** 0.5
    if fmt == "int8":
        return torch.randint(-128, 128, (E, O, H), generator=g, device=DEV).to(torch.int8), s / 74
    w = (torch.randn((E, O, H), generator=g, device=DEV) * 120).clamp(-448, 448)
    return w.to(torch.float8_e4m3fn), s / 120


def reference(x, ids, w, w13, s13, w2, s2):
    """The layer in 64 bits and the bound above, expert by expert."""
    T, H = x.shape
    E, O, _ = w13.shape
    I, K = O // 2, ids.shape[1]
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        A = w13[e].double() * (1.0 if s13 is None else s13[e].double()[:, None])
        B = w2[e].double() * (1.0 if s2 is None else s2[e].double()[:, None])
        X = x[t].double()
        h, dh = X @ A.T, (H + 2) * 2.0 ** -23 * (X.abs() @ A.abs().T)
        g, u, dg, du = h[:, :I], h[:, I:], dh[:, :I], dh[:, I:]
        sl = g * torch.sigmoid(g)                       # |silu'| <= 1.1
        a = sl * u
        da = 1.1 * dg * u.abs() + sl.abs() * du + 1.1 * dg * du + \
            (2.0 ** -16 + 2.0 ** -20) * a.abs() + 2.0 ** -133
        y = a @ B.T
        dy = da @ B.abs().T + (I + 4) * 2.0 ** -23 * ((1.01 * a.abs() + da) @ B.abs().T)
        gate = w[t, k].double()[:, None]
        out.index_add_(0, t, gate * y)
        tol.index_add_(0, t, gate.abs() * (dy + (K + 8) * 2.0 ** -23 * y.abs()))
    return out, tol + 2.0 ** -8 * (out.abs() + tol) + 2.0 ** -133


def handle(api, E, H, I, K, T, fmt):
    code = {"bf16": api.MOE_FORMAT_BF16, "e4m3": api.MOE_FORMAT_FP8_E4M3,
            "int8": api.MOE_FORMAT_INT8}[fmt]
    return api.MoeLayerSmall(E, H, I, K, T, code, DEV)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [33, 40, 44, 48, 56, 64])
def test_layer_hot_expert_with_rings_that_turn(api, fmt, T):
    # every token on expert 5: 4 to 6 stages of 8-bit weights (5 for 44 and 48
    # tokens), 3 to 4 of bf16; about 65 units a CTA and phase 0, half in phase 1
    E, H, I, K = 40, 2048, 1024, 8
    g = gen(T)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    score = torch.rand((T, E), generator=g, device=DEV)
    score[:, 5] = 2.0
    ids = torch.topk(score, K, dim=-1).indices.int().contiguous()
    w = torch.softmax(torch.randn((T, K), generator=g, device=DEV), -1)
    w13, s13 = weights(E, 2 * I, H, fmt, T + 1)
    w2, s2 = weights(E, H, I, fmt, T + 2)
    h = handle(api, E, H, I, K, T, fmt)
    ref, tol = reference(x, ids, w, w13, s13, w2, s2)
    first = None
    for _ in range(6):
        out = torch.full_like(x, float("nan"))
        h.forward(x, ids, w, w13, w2, s13, s2, out=out)
        assert h.get_error() == (0, 0)
        err = (out.double() - ref).abs()
        assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))
        first = out if first is None else first
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,I", [(2048, 1024), (2048, 8192), (272, 144)])  # whole, cut, ragged
def test_layer_keeps_the_second_term_of_the_activations(api, fmt, H, I):
    # W2 subtracts activations that are all near 3, so outputs are small beside what
    # the leading terms leave out (up to 2^-7 each).  Experts of 1, 9 and 54 tokens.
    E, T = 3, 64
    g = gen(H + I)
    d = torch.randint(-15, 16, (E, I), generator=g, device=DEV).float()  # exact in 8 bits
    w13 = torch.zeros((E, 2 * I, H), device=DEV)
    w13[:, :I, 0], w13[:, :I, H - 1], w13[:, I:, 0] = 3.0, d, 1.0
    i = torch.randint(0, I, (E, H), generator=g, device=DEV)
    j = (i + torch.randint(1, I, (E, H), generator=g, device=DEV)) % I
    w2 = torch.zeros((E, H, I), device=DEV)
    w2.scatter_(2, i[:, :, None], 1.0)
    w2.scatter_(2, j[:, :, None], -1.0)
    x = torch.zeros((T, H), device=DEV)
    x[:, 0] = 1.0
    x[:, H - 1] = (1.0 + torch.arange(T, device=DEV) / 64) / 64
    x = x.to(torch.bfloat16)
    ids = torch.full((T, 1), 2, dtype=torch.int32, device=DEV)
    ids[20], ids[3:12] = 0, 1
    w = torch.ones((T, 1), device=DEV)
    one = [None if fmt == "bf16" else torch.ones((E, n), device=DEV) for n in (2 * I, H)]
    kind = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
    h = handle(api, E, H, I, 1, T, fmt)
    out = h.forward(x, ids, w, w13.to(kind), w2.to(kind), *one).double()
    assert h.get_error() == (0, 0)
    # two products of a row are not zero, and sums with zeros are exact
    X = x.double()
    for e in range(E):
        t = (ids[:, 0] == e).nonzero()[:, 0]
        gate = X[t] @ w13[e, :I].double().T             # up is 1, exactly
        a = gate * torch.sigmoid(gate)
        B = w2[e].double()
        da = 1.1 * 4 * 2.0 ** -23 * gate.abs() + (2.0 ** -16 + 2.0 ** -20) * a
        dy = da @ B.abs().T + 4 * 2.0 ** -23 * (1.01 * a) @ B.abs().T
        y = a @ B.T
        tol = dy + 2.0 ** -8 * (y.abs() + dy)
        assert ((out[t] - y).abs() <= tol).all(), (e, float(((out[t] - y).abs() / tol).max()))
        # the leading terms alone would not pass, whatever the token
        lead = a.to(torch.bfloat16).double() @ B.T
        assert ((lead - y).abs() > tol).any(1).all()
