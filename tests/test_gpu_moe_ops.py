"""Router gate, 8-bit integer quantiser and product, and the whole layer for a
few tokens against plain 64-bit (or exact integer) implementations.

Tolerances are counted from roundings: a narrowing to bf16 is off by at most
2^-8 relative, an fp32 operation by 2^-24, a sum of n products in fp32 (in the
tensor cores' own order) by n * 2^-23 of the sum of their magnitudes.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()


@pytest.fixture(scope="module")
def api():
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---- router gate -----------------------------------------------------------------

def gate_ref(logits, K, sigmoid, renorm, scale):
    l = logits.double().cpu().numpy()
    T, E = l.shape
    ids = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    for t in range(T):
        open_ = [e for e in range(E) if l[t, e] > -np.inf]      # (NaN compares false)
        order = sorted(open_, key=lambda e: (-l[t, e], e))[:K]
        if sigmoid:
            s = {e: 1.0 / (1.0 + np.exp(-l[t, e])) for e in order}
        elif order:
            m = l[t, order[0]]
            f = lambda e: 1.0 if l[t, e] == m else np.exp(l[t, e] - m)
            tot = sum(f(e) for e in open_)
            s = {e: f(e) / tot for e in order}
        for k, e in enumerate(order):
            ids[t, k] = e
            w[t, k] = s[e]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale


def check_gate(api, logits, K, sigmoid=0, renorm=True, scale=1.0, **kw):
    ids, w = api.topk_gate(logits, K, sigmoid, renorm, scale, **kw)
    torch.cuda.synchronize()
    rids, rw = gate_ref(logits.reshape(-1, logits.shape[-1]), K, sigmoid, renorm, scale)
    assert np.array_equal(ids.reshape(-1, K).cpu().numpy(), rids)
    # exp (2 ulp) and its argument's rounding, twice; the sum; divisions
    f = logits.double()
    span = float((f[torch.isfinite(f)].max() - f[torch.isfinite(f)].min()).item()) \
        if torch.isfinite(f).any() else 0.0
    tol = (24 + 2 * span + logits.shape[-1] / 32) * 2.0 ** -24
    got = w.reshape(-1, K).double().cpu().numpy()
    assert (np.abs(got - rw) <= tol * np.abs(rw) + 1e-44).all(), np.abs(got - rw).max()
    return ids, w


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 8), (3, 31, 2), (5, 64, 6), (7, 65, 32),
                                   (33, 256, 8), (4, 257, 8), (2, 1000, 3), (3, 1024, 32),
                                   (1025, 160, 6)])
@pytest.mark.parametrize("sigmoid", [0, 1])
def test_gate(api, T, E, K, sigmoid):
    l = torch.randn((T, E), generator=gen(T * E + K), device=DEV) * 2
    for renorm in (True, False):
        check_gate(api, l, K, sigmoid, renorm, 2.5)
        check_gate(api, l.to(torch.bfloat16), K, sigmoid, renorm)  # many equal logits


@pytest.mark.parametrize("T,E,K", [(5001, 256, 8), (6003, 100, 5), (4999, 33, 3), (20005, 20, 8)])
@pytest.mark.parametrize("sigmoid", [0, 1])
def test_gate_many_tokens(api, T, E, K, sigmoid):
    l = torch.randn((T, E), generator=gen(T), device=DEV)
    l[::7, 2:] = -float("inf")                          # fewer open than K
    l[3::11] = -float("inf")
    check_gate(api, l, K, sigmoid, not sigmoid)
    check_gate(api, l.to(torch.bfloat16), K, sigmoid, bool(sigmoid))


@pytest.mark.parametrize("T", [24, 5003])
@pytest.mark.parametrize("E,K", [(256, 8), (200, 1), (128, 7), (64, 3), (12, 8)])
def test_gate_logits_that_differ_in_their_last_bits(api, T, E, K):
    g = gen(T + E + K)
    l = torch.randn((T, E), generator=g, device=DEV)
    last = torch.randint(0, 64, (T, E), generator=g, device=DEV).float() * 2.0 ** -23
    l[0::6] = 1.5 + last[0::6]                          # all of them
    l[1::6] = -(1.5 + last[1::6])
    l[2::6] = torch.where(last[2::6] < 2.0 ** -19, 3.5 + last[2::6], l[2::6])  # some
    l[3::6, E // 2] = l[3::6].max(-1).values            # two at the top, equal
    l[4::6, E // 3] = torch.nextafter(l[4::6].max(-1).values, torch.tensor(9.0, device=DEV))
    # (and a sixth of the rows as they are)
    check_gate(api, l, K)
    check_gate(api, l, K, 1, False)


def test_gate_ties_take_the_lowest_id(api):
    l = torch.zeros((4, 200), device=DEV)
    l[1, 150:] = 1.0
    l[2, ::2] = -0.0
    l[3] = torch.arange(200, device=DEV) % 3
    ids, _ = check_gate(api, l, 8)
    assert ids[0].tolist() == list(range(8))
    assert ids[1].tolist() == list(range(150, 158))
    assert ids[2].tolist() == list(range(8))


@pytest.mark.parametrize("E", [40, 256, 600])
def test_gate_closed_experts(api, E):
    l = torch.randn((6, E), generator=gen(3), device=DEV)
    l[0] = -float("inf")                                # nothing is left
    l[1, 3:] = -float("inf")                            # fewer than K are
    l[2, 5] = float("nan")
    l[3] = float("nan")
    l[4] = torch.finfo(torch.float32).min               # the lowest number is a number
    l[5, ::7] = torch.finfo(torch.float32).max
    for sigmoid in (0, 1):
        ids, w = check_gate(api, l, 8, sigmoid)
        assert ids[0].tolist() == [-1] * 8 and w[0].abs().max() == 0
        assert (ids[1] >= 0).sum() == 3 and (w[1, 3:] == 0).all()
        assert ids[3].tolist() == [-1] * 8


def test_gate_infinite_logits_share(api):
    l = torch.randn((2, 64), generator=gen(4), device=DEV)
    l[0, [9, 30]] = float("inf")
    ids, w = check_gate(api, l, 4)
    assert ids[0, :2].tolist() == [9, 30] and w[0].tolist() == [0.5, 0.5, 0.0, 0.0]


def test_gate_strided_shaped_and_given_outputs(api):
    big = torch.randn((50, 300), generator=gen(5), device=DEV)
    check_gate(api, big[:, 7:7 + 128], 8)               # rows of a wider matrix
    check_gate(api, big.to(torch.bfloat16)[:, 1:130], 8)
    l = torch.randn((4, 6, 96), generator=gen(6), device=DEV)
    ids = torch.empty((4, 6, 5), dtype=torch.int32, device=DEV)
    w = torch.empty((4, 6, 5), device=DEV)
    a, b = check_gate(api, l, 5, out_ids=ids, out_w=w)
    assert a is ids and b is w
    e, f = api.topk_gate(l[:0], 5)
    assert e.shape == (0, 6, 5) and f.shape == (0, 6, 5)


def test_gate_argument_errors(api):
    l = torch.zeros((4, 64), device=DEV)
    with pytest.raises(ValueError):
        api.topk_gate(l.half(), 2)
    with pytest.raises(ValueError):
        api.topk_gate(l.t(), 2)
    with pytest.raises(ValueError):
        api.topk_gate(l, 2, out_ids=torch.empty((4, 2), device=DEV))
    with pytest.raises(api.MoeA2AError):
        api.topk_gate(l, 65)
    with pytest.raises(ValueError):
        api.topk_gate(torch.zeros((4, 64)), 2)


# ---- quantiser ---------------------------------------------------------------------

def quant_ref(x):
    x = x.float().cpu().numpy()
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)
        s = np.where(amax > 0, np.maximum(amax / np.float32(127), np.float32(2.0 ** -126)),
                     np.float32(1)).astype(np.float32)
        q = np.rint(x / s[..., None])
    bad = ~np.isfinite(amax)
    s[bad] = np.nan
    q[bad] = 0
    return q.astype(np.int8), s


def check_quant(api, x, **kw):
    q, s = api.quantize_rows_int8(x, **kw)
    torch.cuda.synchronize()
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)
    return q, s


@pytest.mark.parametrize("rows,H", [(1, 8), (3, 24), (5, 128), (2, 1040), (700, 2048),
                                    (9, 7168), (2, 16384), (3000, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize(api, rows, H, dtype):
    x = torch.randn((rows, H), generator=gen(rows + H), device=DEV)
    x = x * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=gen(1), device=DEV).float())
    check_quant(api, x.to(dtype))


def test_quantize_ties_extremes_and_special_rows(api):
    H = 64
    x = torch.zeros((10, H), device=DEV)
    x[1] = torch.arange(H, device=DEV) - 31.5           # halves, amax 127 below
    x[1, 0] = 127.0
    x[2] = torch.finfo(torch.float32).max
    x[3] = 1e-44                                        # subnormal: the scale's lower end
    x[4, 5] = float("nan")
    x[5, 6] = float("inf")
    x[6] = -3.0
    x[7, 1] = 2.0 ** -126
    x[8] = torch.linspace(-1e30, 1e30, H, device=DEV)
    x[9] = torch.linspace(-1e-33, 1e-33, H, device=DEV)
    q, s = check_quant(api, x)
    assert s[0] == 1.0 and (q[0] == 0).all()
    assert q[1, 1:5].tolist() == [-30, -30, -28, -28]   # -30.5, -29.5, -28.5, -27.5: to even
    assert (q[6] == -127).all() and torch.isnan(s[4]) and torch.isnan(s[5])


def test_quantize_bf16_every_pair_of_significands(api):
    # each bf16 row maximum in a binade with every bf16 value whose code can
    # differ from zero: 128 x 128 significands, ten binades, both signs
    m = np.arange(128, 256).astype(np.float64)
    x = np.ldexp(m[None, :], -np.arange(10)[:, None]).reshape(-1)
    rows = np.minimum(x[None, :], m[:, None])
    rows = np.concatenate([m[:, None], rows, -rows, np.zeros((128, 7))], 1)
    for scale in (1.0, 2.0 ** -110, 2.0 ** 100):
        t = torch.from_numpy((rows * scale).astype(np.float32)).to(DEV)
        assert torch.equal(t.to(torch.bfloat16).float(), t)
        check_quant(api, t.to(torch.bfloat16))
        check_quant(api, t)


def test_quantize_planes_leave_padding_alone(api):
    G, rows, H = 5, 7, 256
    x = torch.randn((G, rows, H), generator=gen(9), device=DEV).to(torch.bfloat16)
    counts = torch.tensor([0, 7, 3, 1, 9], dtype=torch.int32, device=DEV)
    x[2, 3:] = float("nan")                             # never read for a result
    q = torch.full((G, rows, H), 55, dtype=torch.int8, device=DEV)
    s = torch.full((G, rows), 77.0, device=DEV)
    api.quantize_rows_int8(x, counts, q, s)
    torch.cuda.synchronize()
    rq, rs = quant_ref(x)
    for g, c in enumerate([0, 7, 3, 1, 7]):
        assert np.array_equal(q[g, :c].cpu().numpy(), rq[g, :c])
        assert np.array_equal(s[g, :c].cpu().numpy(), rs[g, :c])
        assert (q[g, c:] == 55).all() and (s[g, c:] == 77.0).all()


def test_quantize_strided_rows_and_errors(api):
    big = torch.randn((20, 512), generator=gen(10), device=DEV)
    check_quant(api, big[:, 64:320])
    check_quant(api, big.to(torch.bfloat16)[:, 128:264])
    q, s = api.quantize_rows_int8(big[:0])
    assert q.shape == (0, 512) and s.shape == (0,)
    with pytest.raises(ValueError):
        api.quantize_rows_int8(big.t())
    with pytest.raises(ValueError):
        api.quantize_rows_int8(big.double())
    with pytest.raises(ValueError):
        api.quantize_rows_int8(big, counts=torch.zeros(20, dtype=torch.int32, device=DEV))
    with pytest.raises(api.MoeA2AError):
        api.quantize_rows_int8(torch.zeros((2, 12), device=DEV))
    with pytest.raises(api.MoeA2AError):
        api.quantize_rows_int8(big[:, 1:257])           # rows off 16 bytes


# ---- 8-bit product --------------------------------------------------------------------

def bits(t):
    return t.view(torch.int16)


def gemm_case(G, M, N, H, seed, spread=127):
    g = gen(seed)
    xq = torch.randint(-spread, spread + 1, (G, M, H), generator=g, device=DEV).to(torch.int8)
    wq = torch.randint(-spread, spread + 1, (G, N, H), generator=g, device=DEV).to(torch.int8)
    sx = torch.rand((G, M), generator=g, device=DEV) + 0.01
    sw = torch.rand((G, N), generator=g, device=DEV) * 1e-3 + 1e-5
    return xq, sx, wq, sw


def gemm_ref(xq, sx, wq, sw):
    """Exact integer sums (float64 holds them), then the two fp32 products."""
    dot = torch.bmm(xq.double(), wq.double().transpose(1, 2))
    assert dot.abs().max() <= 2 ** 24
    return ((dot.float() * sx[:, :, None]) * sw[:, None, :]).to(torch.bfloat16)


@pytest.mark.parametrize("G,M,N,H", [
    (1, 1, 1, 16), (1, 1, 128, 128), (1, 16, 7, 144), (1, 17, 130, 256), (1, 64, 1000, 272),
    (1, 129, 257, 1040), (1, 300, 640, 512), (1, 257, 4096, 2048), (3, 40, 200, 384),
    (1, 1000, 3000, 528), (1, 2048, 2304, 1024), (7, 5, 96, 4096), (1, 3, 5000, 7168)])
def test_gemm_exact(api, G, M, N, H):
    xq, sx, wq, sw = gemm_case(G, M, N, H, G + M + N + H, 127 if H <= 1024 else 40)
    h = api.MoeGemmInt8(G, M, N, H, DEV)
    ref = gemm_ref(xq, sx, wq, sw)
    for _ in range(3):                                  # the scratch serves call after call
        out = torch.full((G, M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
        h.gemm(xq, sx, wq, sw, out=out)
        assert h.get_error() == (0, 0)
        assert torch.equal(bits(out), bits(ref))


@pytest.mark.parametrize("G,M,N,H", [(6, 33, 136, 256), (32, 1024, 512, 512), (9, 300, 384, 784),
                                     (64, 16, 256, 128), (1024, 3, 40, 48), (5, 600, 130, 6000)])
def test_gemm_ragged_groups(api, G, M, N, H):
    xq, sx, wq, sw = gemm_case(G, M, N, H, 3)
    counts = torch.randint(0, M + 1, (G,), generator=gen(4), device=DEV).to(torch.int32)
    counts[0], counts[1], counts[2] = 0, M, 1
    out = torch.full((G, M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    h = api.MoeGemmInt8(G, M, N, H, DEV)
    h.gemm(xq, sx, wq, sw, counts, out)
    assert h.get_error() == (0, 0)
    ref = gemm_ref(xq, sx, wq, sw)
    for g, c in enumerate(counts.tolist()):
        assert torch.equal(bits(out[g, :c]), bits(ref[g, :c])), g
        assert torch.isnan(out[g, c:]).all(), g         # padding is left alone


def test_gemm_no_rows_anywhere_and_counts_out_of_range(api):
    G, M, N, H = 4, 20, 64, 64
    xq, sx, wq, sw = gemm_case(G, M, N, H, 5)
    h = api.MoeGemmInt8(G, M, N, H, DEV)
    out = torch.full((G, M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    h.gemm(xq, sx, wq, sw, torch.zeros(G, dtype=torch.int32, device=DEV), out)
    assert h.get_error() == (0, 0) and (out == 3.0).all()
    h.gemm(xq, sx, wq, sw, torch.tensor([-5, 100, 0, 2], dtype=torch.int32, device=DEV), out)
    assert h.get_error() == (0, 0)
    ref = gemm_ref(xq, sx, wq, sw)
    assert (out[0] == 3.0).all() and torch.equal(out[1], ref[1])
    assert torch.equal(out[3, :2], ref[3, :2]) and (out[3, 2:] == 3.0).all()


def test_gemm_all_codes_and_the_largest_sums(api):
    # -128 is a code too; sums past 2^24 round like any fp32 sum
    H = 7168
    xq = torch.full((1, 20, H), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((1, 130, H), -128, dtype=torch.int8, device=DEV)
    xq[0, 1], wq[0, 1] = 127, 127
    xq[0, 2] = torch.arange(H, device=DEV).to(torch.int8)
    wq[0, 2] = torch.arange(H, device=DEV).flip(0).to(torch.int8)
    sx, sw = torch.ones((1, 20), device=DEV), torch.ones((1, 130), device=DEV)
    h = api.MoeGemmInt8(1, 20, 130, H, DEV)
    out = h.gemm(xq, sx, wq, sw).double()
    dot = torch.bmm(xq.double(), wq.double().transpose(1, 2))
    mag = torch.bmm(xq.double().abs(), wq.double().abs().transpose(1, 2))
    assert ((out - dot).abs() <= 2.0 ** -8 * dot.abs() + H * 2.0 ** -23 * mag).all()


def test_gemm_sums_that_cancel(api):
    # partial sums just below 2^24, results of a few units: exact, so nothing of
    # the small parts was lost on the way
    H = 2080
    xq = torch.full((1, 40, H), 127, dtype=torch.int8, device=DEV)
    wq = torch.full((1, 300, H), 127, dtype=torch.int8, device=DEV)
    wq[:, :, H // 2:] = -127                            # 1040 * 127^2 = 2^24 - 3056
    for n in range(300):
        wq[0, n, 3 + n % 500] = 127 - n % 3             # off by 0, 127 and 254
    for m in range(40):
        xq[0, m, H - 1 - m] = 127 - m % 2               # off by 0 and -127 (times -1)
    one = lambda n: torch.ones((1, n), device=DEV)
    out = api.MoeGemmInt8(1, 40, 300, H, DEV).gemm(xq, one(40), wq, one(300))
    ref = torch.bmm(xq.double(), wq.double().transpose(1, 2))
    assert ref.abs().max() <= 256 and torch.equal(out.double(), ref)


def test_gemm_nan_scales_stay_in_their_rows(api):
    xq, sx, wq, sw = gemm_case(1, 30, 200, 256, 6)
    sx[0, 7] = float("nan")
    sw[0, 11] = float("inf")
    out = api.MoeGemmInt8(1, 30, 200, 256, DEV).gemm(xq, sx, wq, sw)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 7] = True
    bad[0, :, 11] = True
    assert torch.isfinite(out[~bad]).all() and torch.isnan(out[0, 7]).all()


def test_gemm_fewer_rows_two_dims_streams_and_errors(api):
    xq, sx, wq, sw = gemm_case(1, 100, 300, 320, 7)
    h = api.MoeGemmInt8(1, 128, 300, 320, DEV)          # prepared for more rows
    ref = gemm_ref(xq, sx, wq, sw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = h.gemm(xq[0], sx[0], wq[0], sw[0], stream=st)
    st.synchronize()
    assert out.shape == (100, 300) and torch.equal(out, ref[0])
    assert h.gemm(xq[:, :0], sx[:, :0], wq, sw).shape == (1, 0, 300)
    with pytest.raises(ValueError):
        h.gemm(xq, sx, wq[:, :, :160], sw)
    with pytest.raises(ValueError):
        h.gemm(xq.transpose(1, 2), sx, wq, sw)
    with pytest.raises(ValueError):
        h.gemm(xq, sx.double(), wq, sw)
    with pytest.raises(api.MoeA2AError):
        h.gemm(*gemm_case(1, 129, 300, 320, 7))
    with pytest.raises(api.MoeA2AError):
        api.MoeGemmInt8(1, 0, 300, 320, DEV)


# ---- past 2^31 elements ----------------------------------------------------------

def test_gate_beyond_32_bits(api):
    T, E = 2200000, 1000
    l = torch.empty((T, E), dtype=torch.bfloat16, device=DEV)
    l[:100].normal_(generator=gen(1))
    l[100:-100].zero_()
    l[-100:].normal_(generator=gen(2))
    ids, w = api.topk_gate(l, 4)
    for part in (slice(0, 100), slice(T - 100, T)):
        rids, rw = gate_ref(l[part], 4, 0, True, 1.0)
        assert np.array_equal(ids[part].cpu().numpy(), rids)
    assert (ids[100:-100] == torch.arange(4, device=DEV)).all()


def test_quantize_beyond_32_bits(api):
    rows, H = 135000, 16384
    x = torch.zeros((rows, H), dtype=torch.bfloat16, device=DEV)
    x[-50:].normal_(generator=gen(3))
    q, s = api.quantize_rows_int8(x)
    rq, rs = quant_ref(x[-50:])
    assert np.array_equal(q[-50:].cpu().numpy(), rq) and np.array_equal(s[-50:].cpu().numpy(), rs)
    assert (s[:-50] == 1).all() and not q[:-50].any()


def test_gemm_beyond_32_bits(api):
    M, N, H = 300000, 8192, 64                          # 2.4 G outputs
    xq, sx, wq, sw = gemm_case(1, M, N, H, 8)
    out = api.MoeGemmInt8(1, M, N, H, DEV).gemm(xq, sx, wq, sw)
    for part in (slice(0, 300), slice(M - 300, M)):
        ref = gemm_ref(xq[:, part].contiguous(), sx[:, part], wq, sw)
        assert torch.equal(bits(out[:, part].contiguous()), bits(ref))


def test_layer_beyond_32_bits(api):
    E, H, I = 64, 7168, 2400                            # W13: 2.2 G weights
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device=DEV)
    for e in (0, E - 1):
        w13[e].normal_(0, H ** -0.5, generator=gen(e))
        w2[e].normal_(0, I ** -0.5, generator=gen(e + 1))
    x = torch.randn((3, H), generator=gen(5), device=DEV).to(torch.bfloat16)
    ids = torch.tensor([[0, E - 1], [E - 1, 5], [7, 0]], dtype=torch.int32, device=DEV)
    w = torch.rand((3, 2), generator=gen(6), device=DEV)
    check_layer(api, (x, ids, w, w13, None, w2, None), "bf16")


# ---- whole layer ------------------------------------------------------------------------

FORMATS = ["bf16", "e4m3", "int8"]


def layer_weights(E, O, H, fmt, seed):
    g = gen(seed)
    if fmt == "bf16":
        return (torch.randn((E, O, H), generator=g, device=DEV) / H ** 0.5).to(torch.bfloat16), None
    s = (torch.rand((E, O), generator=g, device=DEV) + 0.5) / H ** 0.5
    if fmt == "int8":
        w = torch.randint(-128, 128, (E, O, H), generator=g, device=DEV).to(torch.int8)
        return w, s / 74
    w = (torch.randn((E, O, H), generator=g, device=DEV) * 120).clamp(-448, 448)
    w[:, :, ::17] *= 2.0 ** -12                         # among them subnormal codes
    return w.to(torch.float8_e4m3fn), s / 120


def layer_ref(x, ids, w, w13, s13, w2, s2, residual=None):
    """The layer in 64 bits and how far fp32 accumulation, the activations'
    narrowing and the output's may take a result from it."""
    T, H = x.shape
    E, O, _ = w13.shape
    I = O // 2
    X = x.double()
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for t in range(T):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if not 0 <= e < E:
                continue
            A = w13[e].double() * (1.0 if s13 is None else s13[e].double()[:, None])
            B = w2[e].double() * (1.0 if s2 is None else s2[e].double()[:, None])
            h, dh = A @ X[t], (H + 2) * 2.0 ** -23 * (A.abs() @ X[t].abs())
            g, u, dg, du = h[:I], h[I:], dh[:I], dh[I:]
            sl = g * torch.sigmoid(g)
            a = sl * u                                  # |silu'| <= 1.1
            da = 1.1 * dg * u.abs() + sl.abs() * du + 1.1 * dg * du + \
                (2.0 ** -8 + 2.0 ** -20) * a.abs() + 2.0 ** -133
            y = B @ a
            dy = B.abs() @ da + (I + 2) * 2.0 ** -23 * (B.abs() @ (a.abs() + da))
            gate = float(w[t, k])
            out[t] += gate * y
            tol[t] += abs(gate) * (dy + 40 * 2.0 ** -23 * y.abs())
    if residual is not None:
        out += residual.double()
        tol += 2.0 ** -23 * out.abs()
    return out, tol + 2.0 ** -8 * (out.abs() + tol) + 2.0 ** -133


def layer_case(T, E, H, I, K, fmt, seed, absent=0):
    g = gen(seed)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.topk(torch.rand((T, E), generator=g, device=DEV), K, dim=-1).indices.int()
    w = torch.softmax(torch.randn((T, K), generator=g, device=DEV), -1)
    if absent:
        ids[T - absent:] = -1
    w13, s13 = layer_weights(E, 2 * I, H, fmt, seed + 1)
    w2, s2 = layer_weights(E, H, I, fmt, seed + 2)
    return x, ids.contiguous(), w, w13, s13, w2, s2


def layer_handle(api, E, H, I, K, T, fmt):
    code = {"bf16": api.MOE_FORMAT_BF16, "e4m3": api.MOE_FORMAT_FP8_E4M3,
            "int8": api.MOE_FORMAT_INT8}[fmt]
    return api.MoeLayerSmall(E, H, I, K, T, code, DEV)


def check_layer(api, case, fmt, T=None, residual=None, expect=(0, 0), handle=None):
    x, ids, w, w13, s13, w2, s2 = case
    E, H, I, K = w13.shape[0], x.shape[1], w2.shape[2], ids.shape[1]
    h = handle or layer_handle(api, E, H, I, K, T or x.shape[0], fmt)
    out = torch.full_like(x, float("nan"))
    h.forward(x, ids, w, w13, w2, s13, s2, residual=residual, out=out)
    assert h.get_error() == expect
    ref, tol = layer_ref(x, ids, w, w13, s13, w2, s2, residual)
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))
    return h, out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,H,I,K", [
    (1, 1, 16, 16, 1), (1, 8, 128, 64, 2), (2, 4, 144, 80, 3), (3, 16, 256, 192, 4),
    (5, 24, 1424, 720, 4), (16, 8, 512, 256, 2), (17, 40, 272, 112, 8), (33, 12, 640, 48, 5),
    (64, 32, 384, 256, 8), (64, 3, 256, 128, 3), (1, 64, 2048, 768, 8), (4, 300, 128, 32, 32)])
def test_layer(api, fmt, T, E, H, I, K):
    case = layer_case(T, E, H, I, K, fmt, T + E + H)
    h, out = check_layer(api, case, fmt)
    x, ids, w, w13, s13, w2, s2 = case
    for _ in range(4):                                  # same call, same bits
        again = h.forward(x, ids, w, w13, w2, s13, s2)
        assert torch.equal(bits(again), bits(out))
    assert h.get_error() == (0, 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hot", [False, True])
def test_layer_at_its_limits(api, fmt, hot):
    # 64 tokens, 1024 experts, top-32: the longest lists, and (hot) every token on
    # the same 32 experts, the fewest stages
    x, ids, w, w13, s13, w2, s2 = layer_case(64, 1024, 64, 16, 32, fmt, 91)
    if hot:
        ids[:] = torch.arange(992, 1024, dtype=torch.int32, device=DEV)
    check_layer(api, (x, ids, w, w13, s13, w2, s2), fmt)


def test_layer_widest(api):
    check_layer(api, layer_case(2, 2, 16384, 16384, 1, "int8", 92), "int8")


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_residual_absent_tokens_and_larger_handle(api, fmt):
    case = layer_case(9, 10, 320, 96, 3, fmt, 21, absent=4)
    res = torch.randn((9, 320), generator=gen(22), device=DEV).to(torch.bfloat16)
    h, out = check_layer(api, case, fmt, T=64, residual=res)
    assert torch.equal(out[5:], res[5:])                # no expert: the residual alone
    _, out = check_layer(api, case, fmt, handle=h)
    assert (out[5:] == 0).all()
    x, ids, w, w13, s13, w2, s2 = case
    first = h.forward(x, ids, w, w13, w2, s13, s2, residual=res)
    same = res.clone()                                  # in place
    h.forward(x, ids, w, w13, w2, s13, s2, residual=same, out=same)
    assert torch.equal(bits(first), bits(same))


def test_layer_no_expert_at_all(api):
    x, ids, w, w13, s13, w2, s2 = layer_case(6, 8, 256, 64, 2, "bf16", 31)
    ids.fill_(-1)
    h = layer_handle(api, 8, 256, 64, 2, 6, "bf16")
    out = torch.full_like(x, 5.0)
    h.forward(x, ids, w, w13, w2, out=out)
    assert h.get_error() == (0, 0) and (out == 0).all()
    h.forward(x, ids, w, w13, w2, residual=x, out=out)
    assert h.get_error() == (0, 0) and torch.equal(out, x)
    assert h.forward(x[:0], ids[:0], w[:0], w13, w2).shape == (0, 256)


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_repeated_experts_and_bad_ids(api, fmt):
    x, ids, w, w13, s13, w2, s2 = layer_case(7, 5, 256, 64, 4, fmt, 41)
    ids[0] = 2                                          # all four the same
    ids[1] = torch.tensor([1, 3, 1, 3], device=DEV)
    ids[2] = torch.tensor([-1, 4, -1, 4], device=DEV)
    check_layer(api, (x, ids, w, w13, s13, w2, s2), fmt)
    ids[3, 1], ids[4, 0] = 5, -7                        # no such experts: skipped, flagged
    h, _ = check_layer(api, (x, ids, w, w13, s13, w2, s2), fmt,
                       expect=(api.MOE_ERR_ROUTING, api.MOE_DEVICE_FLAG_BAD_EXPERT_ID))
    ids[3, 1], ids[4, 0] = 0, 0
    check_layer(api, (x, ids, w, w13, s13, w2, s2), fmt, handle=h)   # works on


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_hot_expert_and_nan_token(api, fmt):
    T, E, H, I, K = 64, 6, 256, 128, 2
    x, ids, w, w13, s13, w2, s2 = layer_case(T, E, H, I, K, fmt, 51)
    ids[:, 0], ids[:, 1] = 3, 0                         # two experts take every token
    h, out = check_layer(api, (x, ids, w, w13, s13, w2, s2), fmt)
    x[10] = float("nan")
    poisoned = h.forward(x, ids, w, w13, w2, s13, s2)
    assert torch.isnan(poisoned[10]).all()
    keep = [t for t in range(T) if t != 10]
    assert torch.equal(bits(poisoned[keep]), bits(out[keep]))


def test_layer_nan_weights(api):
    x, ids, w, w13, s13, w2, s2 = layer_case(4, 4, 128, 64, 2, "e4m3", 61)
    ids[0], ids[1] = torch.tensor([0, 1], device=DEV), torch.tensor([1, 2], device=DEV)
    ids[2], ids[3] = torch.tensor([2, 3], device=DEV), torch.tensor([3, 1], device=DEV)
    raw = w2.view(torch.uint8)
    raw[0, 5, 7] = 0x7F                                 # expert 0, channel 5: NaN codes
    raw[0, 9, 30] = 0xFF
    h = layer_handle(api, 4, 128, 64, 2, 4, "e4m3")
    out = h.forward(x, ids, w, w13, raw, s13, s2)       # codes as bytes are taken too
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[0, [5, 9]] = True
    assert torch.equal(bad, want)


def test_layer_in_a_graph_and_on_a_stream(api):
    T, E, H, I, K = 8, 16, 512, 256, 4
    x, ids, w, w13, s13, w2, s2 = layer_case(T, E, H, I, K, "int8", 71)
    h = layer_handle(api, E, H, I, K, T, "int8")
    eager = h.forward(x, ids, w, w13, w2, s13, s2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = h.forward(x, ids, w, w13, w2, s13, s2, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(bits(eager), bits(other))
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.forward(x, ids, w, w13, w2, s13, s2, out=out)
    for seed in (72, 73):
        nx, nids, nw = layer_case(T, E, H, I, K, "int8", seed)[:3]
        x.copy_(nx), ids.copy_(nids), w.copy_(nw)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert h.get_error() == (0, 0)
        assert torch.equal(bits(got), bits(h.forward(x, ids, w, w13, w2, s13, s2)))


def test_layer_argument_errors(api):
    x, ids, w, w13, s13, w2, s2 = layer_case(4, 4, 128, 64, 2, "int8", 81)
    h = layer_handle(api, 4, 128, 64, 2, 4, "int8")
    with pytest.raises(ValueError):
        h.forward(x, ids, w, w13, w2)                   # scales are missing
    with pytest.raises(ValueError):
        h.forward(x, ids.long(), w, w13, w2, s13, s2)
    with pytest.raises(ValueError):
        h.forward(x, ids, w, w13.to(torch.bfloat16), w2, s13, s2)
    with pytest.raises(ValueError):
        h.forward(x, ids, w, w13[:, :100], w2, s13, s2)
    with pytest.raises(ValueError):
        h.forward(x.t().contiguous().t(), ids, w, w13, w2, s13, s2)
    with pytest.raises(api.MoeA2AError):
        h.forward(x.repeat(2, 1), ids.repeat(2, 1), w.repeat(2, 1), w13, w2, s13, s2)
    with pytest.raises(api.MoeA2AError):
        api.MoeLayerSmall(4, 128, 60, 2, 4, api.MOE_FORMAT_INT8, DEV)
    with pytest.raises(api.MoeA2AError):
        api.MoeLayerSmall(4, 128, 64, 2, 65, api.MOE_FORMAT_INT8, DEV)
