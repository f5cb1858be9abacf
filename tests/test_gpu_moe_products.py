"""The block quantiser, the 8-bit product with block scales, and the experts'
products over ragged rows with their gradients, against 64-bit implementations.

Most inputs are small integers (and powers of two as scales): every product and
every partial sum is then exact in fp32 in any order (all stay below 2^24), so
the result is the exact sum rounded once, and outputs have to be equal.  Normal
values are compared with tolerances counted from roundings: a narrowing to bf16
is off by at most 2^-8 relative, an fp32 operation by 2^-24, a sum of n products
in fp32 (in the tensor cores' own order) by n * 2^-23 of the sum of magnitudes.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"
BF, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


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


def ints(shape, most, g):
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(BF)


def blocks(n):
    return (n + 127) // 128


def offsets_of(counts, first=0):
    o = np.concatenate([[0], np.cumsum(counts)]) + first
    return torch.tensor(o, dtype=torch.int32, device=DEV)


def same(a, b):
    """Equal, NaN in the same places."""
    return torch.equal(torch.nan_to_num(a.float(), nan=7e30), torch.nan_to_num(b.float(), nan=7e30))


# ---- block quantiser ---------------------------------------------------------------

def quant_ref(x, b):
    """Codes and scales from numpy's binary32 (division is correctly rounded)."""
    x = x.float().cpu().numpy()
    R, H = x.shape
    pad = np.zeros(((R + b - 1) // b * b, blocks(H) * 128), np.float32)
    pad[:R, :H] = np.abs(x)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = pad.reshape(-1, b, blocks(H), 128).max((1, 3))
        s = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126))
        s = np.where(amax == 0, np.float32(1), s)
        s[~np.isfinite(amax)] = np.nan
        each = np.repeat(np.repeat(s, b, 0)[:R], 128, 1)[:, :H]
        q = np.where(np.isnan(each), np.float32(0), x / each)
    q = torch.from_numpy(np.clip(q, -448, 448).astype(np.float32)).to(F8)
    return q, torch.from_numpy(s)


def check_quant(x, b, q, s):
    torch.cuda.synchronize()
    rq, rs = quant_ref(x.reshape(-1, x.shape[-1]), b)
    assert same(s.reshape(rs.shape).cpu(), rs)
    assert torch.equal(q.reshape(rq.shape).view(torch.uint8).cpu(), rq.view(torch.uint8))


@pytest.mark.parametrize("rows,H", [(1, 16), (1, 128), (3, 144), (5, 256), (127, 1040), (128, 128),
                                    (129, 272), (300, 7168), (1000, 48)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("b", [1, 128])
def test_quantize(api, rows, H, dtype, b):
    g = gen(rows * H + b)
    x = torch.randn((rows, H), generator=g, device=DEV)
    x = (x * torch.exp(2 * torch.randn((rows, 1), generator=g, device=DEV))).to(dtype)
    x[rows // 2, : H // 2] = 0
    check_quant(x, b, *api.quantize_blocks_fp8(x, b))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("b", [1, 128])
def test_quantize_extremes(api, dtype, b):
    x = torch.randn((384, 512), generator=gen(1), device=DEV).to(dtype)
    x[0:128, 0:128] = 0                                  # nothing
    x[1, 200] = float("nan")
    x[130, 5] = float("inf")
    x[131, 300] = -float("inf")
    x[256:, 0:128] = torch.finfo(dtype).max              # the largest number is a number
    x[256:, 128:256] = torch.finfo(dtype).tiny * 2       # the scale at its floor
    x[256:, 256:384] = -0.0
    if dtype is F32:
        x[256:, 384:] *= 1e-39                           # subnormal
    check_quant(x, b, *api.quantize_blocks_fp8(x, b))


def test_quantize_every_pair_of_bf16_significands(api):
    """A block's largest value against every value below it down to 2^-23 of it (smaller
    ones have code 0), maxima of 128 significands, with and without scaled quotients."""
    small = torch.arange(128, 256, device=DEV).float()
    below = (small * torch.exp2(-torch.arange(24, device=DEV).float())[:, None]).reshape(-1)
    for power in (0, -100, 110):
        for m in range(128, 256):
            v = below[below <= m]
            v = torch.nn.functional.pad(v, (0, -len(v) % 127)).view(-1, 127)
            v = torch.cat([v, torch.full((len(v), 1), float(m), device=DEV)], 1)
            v[:, ::2] *= -1
            x = (v * 2.0 ** power).to(BF)
            assert torch.equal(x.float(), v * 2.0 ** power)
            check_quant(x, 1, *api.quantize_blocks_fp8(x))


def test_quantize_planes_strides_and_buffers(api):
    g = gen(2)
    x = torch.randn((4, 37, 272), generator=g, device=DEV).to(BF)
    q = torch.full(x.shape, 3, dtype=torch.uint8, device=DEV)
    s = torch.full((4, 37, 3), -5.0, device=DEV)
    counts = torch.tensor([0, 37, 9, 1], dtype=torch.int32, device=DEV)
    got = api.quantize_blocks_fp8(x, counts=counts, out=q, scale=s)
    assert got[0] is q and got[1] is s
    rq, rs = quant_ref(x.reshape(-1, 272), 1)
    rq, rs = rq.view(torch.uint8).reshape(x.shape), rs.reshape(s.shape)
    for e, c in enumerate(counts.tolist()):
        assert torch.equal(q[e, :c].cpu(), rq[e, :c]) and torch.equal(s[e, :c].cpu(), rs[e, :c])
        assert (q[e, c:] == 3).all() and (s[e, c:] == -5).all()
    wide = torch.randn((50, 512), generator=g, device=DEV)
    part = wide[:, 128:400]                              # rows 512 apart
    for b in (1, 128):
        check_quant(part, b, *api.quantize_blocks_fp8(part, b))
    deep = torch.randn((3, 130, 144), generator=g, device=DEV).to(BF)
    q, s = api.quantize_blocks_fp8(deep, 128)
    assert s.shape == (3, 2, 2)
    for e in range(3):
        check_quant(deep[e], 128, q[e], s[e])
    for shape in ((0, 64), (2, 0, 64)):
        q, s = api.quantize_blocks_fp8(torch.empty(shape, device=DEV))
        assert q.shape == shape and s.shape == (*shape[:-1], 1)


# ---- 8-bit product ------------------------------------------------------------------

def fp8_inputs(lead, G, rows, N, H, g, exact=True):
    """Integer codes up to 4 and powers of two as scales, or normal values."""
    if exact:
        xq, wq = ints((*lead, rows, H), 4, g).to(F8), ints((G, N, H), 4, g).to(F8)
        two = lambda shape: torch.exp2(torch.randint(-2, 3, shape, generator=g, device=DEV).float())
    else:
        xq = (torch.randn((*lead, rows, H), generator=g, device=DEV) * 100).clamp(-448, 448).to(F8)
        wq = (torch.randn((G, N, H), generator=g, device=DEV) * 100).clamp(-448, 448).to(F8)
        two = lambda shape: torch.rand(shape, generator=g, device=DEV) * 0.01 + 1e-3
    return xq, two((*lead, rows, blocks(H))), wq, two((G, blocks(N), blocks(H)))


def fp8_ref(xq, sx, wq, sw):
    """One group in 64 bits: the product and the sum of the magnitudes."""
    N, H = wq.shape
    x = xq.double() * sx.double().repeat_interleave(128, -1)[:, :H]
    w = wq.double() * sw.double().repeat_interleave(128, -1)[:, :H].repeat_interleave(128, 0)[:N]
    return x @ w.T, x.abs() @ w.abs().T


SIZES = [(1, 1, 16), (1, 256, 128), (3, 130, 144), (16, 1000, 1040), (17, 129, 384), (64, 512, 512),
         (100, 264, 2048), (255, 70, 640), (80, 144, 256), (81, 144, 256), (256, 256, 128), (257, 513, 272), (700, 300, 1024)]


@pytest.mark.parametrize("rows,N,H", SIZES)
def test_fp8_dense(api, rows, N, H):
    # |sum| <= 1024 * 4 * 4 * 2^4 = 2^18 in steps of 2^-4 (H <= 2048: 2^19): exact
    xq, sx, wq, sw = fp8_inputs((1,), 1, rows, N, H, gen(rows + N + H))
    out = api.MoeGemmFp8(1, rows, N, H, DEV).gemm(xq, sx, wq, sw)
    ref, _ = fp8_ref(xq[0], sx[0], wq[0], sw[0])
    assert torch.equal(out[0], ref.to(BF))
    again = api.MoeGemmFp8(1, rows, N, H, DEV).gemm(xq[0].view(torch.uint8), sx[0], wq[0], sw[0])
    assert torch.equal(again, out[0])


@pytest.mark.parametrize("rows,N,H", [(5, 700, 2064), (300, 900, 4096), (2000, 1500, 1024)])
def test_fp8_normal_values(api, rows, N, H):
    xq, sx, wq, sw = fp8_inputs((1,), 1, rows, N, H, gen(rows), exact=False)
    out = api.MoeGemmFp8(1, rows, N, H, DEV).gemm(xq, sx, wq, sw)
    ref, mag = fp8_ref(xq[0], sx[0], wq[0], sw[0])
    # a block's 128 products; its scales' product; a fused multiply-add a block
    tol = 2.0 ** -8 * ref.abs() + (128 + 1 + blocks(H)) * 2.0 ** -23 * mag
    assert ((out[0].double() - ref).abs() <= tol).all()
    # the rounding to bf16 is at most 2^-8 of each value: so is the norm, the sums' share
    # is far below it for normal values
    assert (out[0].double() - ref).norm() <= 2.0 ** -8 * ref.norm()


COUNTS = [[0], [1], [0, 0, 0], [300], [5, 0, 17, 1], [256, 0, 255, 257, 31],
          [0, 700, 3, 64, 64, 1, 0, 0, 90], [2] * 40, [0] * 100 + [33] + [0] * 100]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "%dx%d" % (len(c), max(c)))
@pytest.mark.parametrize("N,H", [(72, 144), (520, 400)])
def test_fp8_groups(api, counts, N, H):
    G, total = len(counts), sum(counts)
    g = gen(total + N)
    handle = api.MoeGemmFp8(G, total + 9, N, H, DEV)
    # rows one group after another, some in front and behind that belong to none
    rows = total + 8
    xq, sx, wq, sw = fp8_inputs((), G, rows, N, H, g)
    off = offsets_of(counts, 3)
    none = torch.ones(rows, dtype=torch.bool, device=DEV)
    none[3:3 + total] = False
    xq.view(torch.uint8)[none] = 0x7f                    # NaN
    sx[none] = float("nan")
    out = torch.full((rows, N), 7.0, dtype=BF, device=DEV)
    assert handle.gemm(xq, sx, wq, sw, offsets=off, out=out) is out
    want = torch.full_like(out, 7.0)
    for e in range(G):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            want[a:b] = fp8_ref(xq[a:b], sx[a:b], wq[e], sw[e])[0].to(BF)
    assert torch.equal(out, want)
    # planes with counts (a count past the plane is the plane)
    M = max(1, max(counts))
    xq, sx, wq, sw = fp8_inputs((G,), G, M, N, H, g)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    cnt[cnt == M] = M + 5
    out = torch.full((G, M, N), 7.0, dtype=BF, device=DEV)
    handle.gemm(xq, sx, wq, sw, counts=cnt, out=out)
    want = torch.full_like(out, 7.0)
    for e, c in enumerate(counts):
        want[e, :c] = fp8_ref(xq[e, :c], sx[e, :c], wq[e], sw[e])[0].to(BF)
    assert torch.equal(out, want)
    assert handle.get_error() == (api.MOE_OK, 0)


@pytest.mark.parametrize("seed,N,H", [(1, 1024, 256), (2, 1096, 720), (3, 520, 2048), (4, 1003, 640)])
def test_fp8_many_tiles_of_every_width(api, seed, N, H):
    """More tiles than SMs, groups of no token up to several tiles, in one call."""
    rng = np.random.default_rng(seed)
    G, M = 40, 600
    counts = np.concatenate([rng.integers(0, 140, 20), rng.integers(0, M + 1, 20)])
    counts[[3, 20, 39]] = 0
    rng.shuffle(counts)
    g = gen(seed)
    handle = api.MoeGemmFp8(G, M, N, H, DEV)
    xq, sx, wq, sw = fp8_inputs((G,), G, M, N, H, g)
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    want = torch.full((G, M, N), 7.0, dtype=BF, device=DEV)
    for e, c in enumerate(counts.tolist()):
        want[e, :c] = fp8_ref(xq[e, :c], sx[e, :c], wq[e], sw[e])[0].to(BF)
    for _ in range(3):
        out = torch.full((G, M, N), 7.0, dtype=BF, device=DEV)
        handle.gemm(xq, sx, wq, sw, counts=cnt, out=out)
        assert torch.equal(out, want)
    assert handle.get_error() == (api.MOE_OK, 0)


def test_fp8_takes_what_the_quantiser_gives(api):
    rows, N, H = 70, 300, 1040
    g = gen(9)
    x = torch.randn((rows, H), generator=g, device=DEV)
    w = torch.randn((N, H), generator=g, device=DEV).to(BF)
    xq, sx = api.quantize_blocks_fp8(x)
    wq, sw = api.quantize_blocks_fp8(w, 128)
    out = api.MoeGemmFp8(1, rows, N, H, DEV).gemm(xq, sx, wq, sw)
    ref = x.double() @ w.double().T
    # a code is off by at most 2^-4 of its value (2^-10 of a scale below the smallest
    # normal code): products by 2 * 2^-4 + 2^-8 and a little
    sxe = sx.double().repeat_interleave(128, 1)[:, :H]
    swe = sw.double().repeat_interleave(128, 1)[:, :H].repeat_interleave(128, 0)[:N]
    ex, ew = x.double().abs() * 2.0 ** -4 + sxe * 2.0 ** -10, w.double().abs() * 2.0 ** -4 + swe * 2.0 ** -10
    tol = ex @ (w.double().abs() + ew).T + x.double().abs() @ ew.T
    mag = (x.double().abs() + ex) @ (w.double().abs() + ew).T
    assert ((out.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -15 * mag).all()


def test_fp8_a_nan_scale_or_code_stays_in_its_row(api):
    rows, N, H = 40, 200, 256
    xq, sx, wq, sw = fp8_inputs((1,), 1, rows, N, H, gen(4))
    clean = api.MoeGemmFp8(1, rows, N, H, DEV).gemm(xq, sx, wq, sw)
    sx[0, 7, 1] = float("nan")
    xq.view(torch.uint8)[0, 9, 3] = 0x7f
    out = api.MoeGemmFp8(1, rows, N, H, DEV).gemm(xq, sx, wq, sw)
    assert out[0, 7].isnan().all() and out[0, 9].isnan().all()
    keep = [r for r in range(rows) if r not in (7, 9)]
    assert torch.equal(out[0, keep], clean[0, keep])


# ---- products over ragged rows, and gradients ------------------------------------------

def ragged(counts, N, H, g, first=2, behind=5):
    """Integers, with NaN in the rows of no expert."""
    total = sum(counts)
    rows = first + total + behind
    x, dy = ints((rows, H), 3, g), ints((rows, N), 3, g)
    w = ints((len(counts), N, H), 3, g)
    for t in (x, dy):
        t[:first] = float("nan")
        t[first + total:] = float("nan")
    return x, dy, w, offsets_of(counts, first)


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "%dx%d" % (len(c), max(c)))
@pytest.mark.parametrize("N,H", [(8, 8), (72, 136), (264, 520), (128, 64), (520, 264), (72, 128),
                                 (264, 384), (40, 1152)])
def test_ragged(api, counts, N, H):
    G = len(counts)
    x, dy, w, off = ragged(counts, N, H, gen(sum(counts) + N + H))
    rows = x.shape[0]
    handle = api.MoeGemmRagged(G, rows, N, H, DEV)
    y = torch.full((rows, N), 7.0, dtype=BF, device=DEV)
    dx = torch.full((rows, H), 7.0, dtype=BF, device=DEV)
    wy, wx = torch.full_like(y, 7.0), torch.full_like(dx, 7.0)
    dw = torch.zeros((G, N, H), dtype=torch.float64, device=DEV)
    for e in range(G):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            wy[a:b] = (x[a:b].double() @ w[e].double().T).to(BF)
            wx[a:b] = (dy[a:b].double() @ w[e].double()).to(BF)
            dw[e] = dy[a:b].double().T @ x[a:b].double()
    assert handle.forward(x, w, off, out=y) is y
    assert torch.equal(y, wy)
    assert handle.input_grad(dy, w, off, out=dx) is dx
    assert torch.equal(dx, wx)
    assert torch.equal(handle.weight_grad(dy, x, off), dw.to(BF))
    assert torch.equal(handle.weight_grad(dy, x, off, dtype=F32), dw.float())
    main = torch.full((G, N, H), 0.5, device=DEV)
    for turn in (1, 2):
        assert handle.weight_grad(dy, x, off, out=main, accumulate=True) is main
        assert torch.equal(main, (dw * turn + 0.5).float())
    assert handle.get_error() == (api.MOE_OK, 0)


@pytest.mark.parametrize("N", [1, 7, 129, 255])
def test_ragged_forward_odd_channels(api, N):
    counts, H = [3, 0, 40, 300], 72
    x, _, w, off = ragged(counts, N, H, gen(N))
    rows = x.shape[0]
    room = torch.full((rows * N + 1,), 7.0, dtype=BF, device=DEV)
    for at in (0, 1):                                    # on a word, and off it
        out = room[at:at + rows * N].view(rows, N)
        out.fill_(7.0)
        api.MoeGemmRagged(4, rows, N, H, DEV).forward(x, w, off, out=out)
        want = torch.full_like(out, 7.0)
        for e in range(4):
            a, b = int(off[e]), int(off[e + 1])
            want[a:b] = (x[a:b].double() @ w[e].double().T).to(BF)
        assert torch.equal(out, want)


@pytest.mark.parametrize("counts", [[2048], [1, 5000, 700], [4000] * 3])
def test_ragged_long(api, counts):
    """Long sums and more tiles than a wave; normal values."""
    G, N, H = len(counts), 1032, 1544
    g = gen(len(counts))
    rows = sum(counts)
    x, dy = torch.randn((rows, H), generator=g, device=DEV).to(BF), \
        torch.randn((rows, N), generator=g, device=DEV).to(BF)
    w = torch.randn((G, N, H), generator=g, device=DEV).to(BF)
    off = offsets_of(counts)
    handle = api.MoeGemmRagged(G, rows, N, H, DEV)
    y, dx = handle.forward(x, w, off), handle.input_grad(dy, w, off)
    dw, dw32 = handle.weight_grad(dy, x, off), handle.weight_grad(dy, x, off, dtype=F32)
    for e in range(G):
        a, b = int(off[e]), int(off[e + 1])
        for got, p, q in ((y[a:b], x[a:b], w[e].T), (dx[a:b], dy[a:b], w[e]),
                          (dw[e], dy[a:b].T, x[a:b]), (dw32[e], dy[a:b].T, x[a:b])):
            p, q = p.double(), q.double()
            ref, mag = p @ q, p.abs() @ q.abs()
            k = p.shape[1]
            narrow = 2.0 ** -8 if got.dtype is BF else 0.0
            assert ((got.double() - ref).abs() <= narrow * ref.abs() + k * 2.0 ** -23 * mag).all()
            # runs of 512 products by truncation, each sum of runs to nearest: far below
            # 2^-8 (and for fp32 below half of 2^-16) of the norm
            far = (got.double() - ref).norm() / ref.norm()
            assert far <= (2.0 ** -8 if got.dtype is BF else 2.0 ** -17)


@pytest.mark.parametrize("seed,N,H", [(1, 776, 520), (2, 520, 640), (3, 1032, 384)])
def test_ragged_many_tiles_of_every_width(api, seed, N, H):
    rng = np.random.default_rng(seed)
    G = 37
    counts = np.concatenate([rng.integers(0, 70, 20), rng.integers(0, 900, 17)])
    counts[[0, 19, 36]] = 0
    rng.shuffle(counts)
    x, dy, w, off = ragged(counts.tolist(), N, H, gen(seed))
    handle = api.MoeGemmRagged(G, x.shape[0], N, H, DEV)
    y, dx = handle.forward(x, w, off), handle.input_grad(dy, w, off)
    dw, dw32 = handle.weight_grad(dy, x, off), handle.weight_grad(dy, x, off, dtype=F32)
    for e in range(G):
        a, b = int(off[e]), int(off[e + 1])
        assert torch.equal(y[a:b], (x[a:b].double() @ w[e].double().T).to(BF))
        assert torch.equal(dx[a:b], (dy[a:b].double() @ w[e].double()).to(BF))
        ref = dy[a:b].double().T @ x[a:b].double()
        assert torch.equal(dw[e], ref.to(BF)) and torch.equal(dw32[e], ref.float())
    assert handle.get_error() == (api.MOE_OK, 0)


def test_ragged_gradients_against_differences(api):
    """The sum over y of a chosen dy changes by dx and dW as the inputs do: the map is
    bilinear, so whole steps give the derivative exactly (integers)."""
    counts, N, H = [9, 0, 70], 24, 40
    g = gen(6)
    x, dy, w, off = ragged(counts, N, H, g, 0, 0)
    handle = api.MoeGemmRagged(3, 79, N, H, DEV)
    f = lambda x, w: (handle.forward(x, w, off).double() * dy.double()).sum().item()
    dx, dw = handle.input_grad(dy, w, off), handle.weight_grad(dy, x, off, dtype=F32)
    x, w = (x / 2).round(), (w / 2).round()              # keep |y| <= 40 * 4 < 256: exact in bf16
    dy = dy.clamp(-1, 1)
    dx, dw = handle.input_grad(dy, w, off), handle.weight_grad(dy, x, off, dtype=F32)
    for m, h in ((0, 0), (8, 39), (9, 3), (78, 17)):
        x2 = x.clone()
        x2[m, h] += 1
        assert f(x2, w) - f(x, w) == dx[m, h].item()
    for e, n, h in ((0, 0, 0), (0, 23, 39), (1, 5, 5), (2, 11, 30)):
        w2 = w.clone()
        w2[e, n, h] += 1
        assert f(x, w2) - f(x, w) == dw[e, n, h].item()


def test_a_nan_stays_with_its_expert(api):
    counts, N, H = [30, 70, 5, 64], 72, 200
    x, dy, w, off = ragged(counts, N, H, gen(8))
    handle = api.MoeGemmRagged(4, x.shape[0], N, H, DEV)
    clean = [handle.forward(x, w, off), handle.input_grad(dy, w, off), handle.weight_grad(dy, x, off)]
    lo, hi = int(off[1]), int(off[2])
    x[lo], x[hi - 1], dy[lo], dy[hi - 1] = (float("nan"),) * 4
    got = [handle.forward(x, w, off), handle.input_grad(dy, w, off), handle.weight_grad(dy, x, off)]
    for c, o in zip(clean[:2], got[:2]):
        assert o[lo].isnan().all() and o[hi - 1].isnan().all()
        for a, b in ((int(off[0]), lo), (lo + 1, hi - 1), (hi, int(off[4]))):
            assert torch.equal(o[a:b], c[a:b])
    assert got[2][1].isnan().all()
    for e in (0, 2, 3):
        assert torch.equal(got[2][e], clean[2][e])


def test_offsets_out_of_range_are_clamped(api):
    counts, N, H = [4, 6, 5], 16, 24
    x, dy, w, _ = ragged(counts, N, H, gen(3), 0, 0)
    handle = api.MoeGemmRagged(3, 15, N, H, DEV)
    bad = torch.tensor([-(1 << 31), 4, 2, (1 << 31) - 1], dtype=torch.int32, device=DEV)
    y = torch.full((15, N), 7.0, dtype=BF, device=DEV)
    dw = handle.weight_grad(dy, x, bad)
    # group 0: rows 0..3; group 1 would end before it begins: none; group 2: rows 2..14
    assert torch.equal(dw[1], torch.zeros_like(dw[1]))
    assert torch.equal(dw[2], (dy[2:].double().T @ x[2:].double()).to(BF))
    handle.forward(x, w, torch.tensor([1, 1, 99, 99], dtype=torch.int32, device=DEV), out=y)
    assert (y[0] == 7).all() and torch.equal(y[1:], (x[1:].double() @ w[1].double().T).to(BF))


# ---- calls in a program -----------------------------------------------------------------

def test_no_rows(api):
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    handle = api.MoeGemmRagged(2, 4, 16, 24, DEV)
    x, dy = torch.empty((0, 24), dtype=BF, device=DEV), torch.empty((0, 16), dtype=BF, device=DEV)
    w = ints((2, 16, 24), 3, gen(1))
    assert handle.forward(x, w, off).shape == (0, 16)
    assert handle.input_grad(dy, w, off).shape == (0, 24)
    dw = torch.ones((2, 16, 24), device=DEV)
    handle.weight_grad(dy, x, off, out=dw, accumulate=True)
    assert (dw == 1).all()
    assert (handle.weight_grad(dy, x, off, out=dw) == 0).all()


def test_calls_follow_one_another_on_one_scratch(api):
    """Many shapes through one handle's scratch, results the same each time."""
    G, N, H = 5, 264, 776
    handle = api.MoeGemmRagged(G, 900, N, H, DEV)
    firsts = []
    for turn in range(3):
        for i, counts in enumerate(([1, 0, 2, 0, 3], [900, 0, 0, 0, 0], [100, 200, 300, 100, 7])):
            g = gen(i)
            x, dy = (torch.randn((sum(counts), n), generator=g, device=DEV).to(BF) for n in (H, N))
            w = torch.randn((G, N, H), generator=g, device=DEV).to(BF)
            off = offsets_of(counts)
            got = [handle.forward(x, w, off), handle.input_grad(dy, w, off),
                   handle.weight_grad(dy, x, off, dtype=F32)]
            if turn == 0:
                firsts.append(got)
            assert all(torch.equal(a, b) for a, b in zip(got, firsts[i]))


def test_captured_and_replayed_with_new_contents(api):
    counts = [7, 0, 130, 64]
    N, H = 136, 264
    rows, G = 210, 4
    handle = api.MoeGemmRagged(G, rows, N, H, DEV)
    eight = api.MoeGemmFp8(G, rows, N, 272, DEV)
    x, dy, w, off = ragged(counts, N, H, gen(5), 0, 9)
    xq, sx, wq, sw = fp8_inputs((), G, rows, N, 272, gen(6))
    y, dx = torch.zeros((rows, N), dtype=BF, device=DEV), torch.zeros((rows, H), dtype=BF, device=DEV)
    dw, y8 = torch.zeros((G, N, H), device=DEV), torch.zeros((rows, N), dtype=BF, device=DEV)

    def step():
        handle.forward(x, w, off, out=y)
        handle.input_grad(dy, w, off, out=dx)
        handle.weight_grad(dy, x, off, out=dw)
        eight.gemm(xq, sx, wq, sw, offsets=off, out=y8)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, counts in ((11, [100, 1, 0, 30]), (12, [0, 0, 0, 210]), (13, [64, 64, 64, 0])):
        nx, ndy, nw, noff = ragged(counts, N, H, gen(seed), 0, rows - sum(counts))
        for t, n in zip((x, dy, w, off), (nx, ndy, nw, noff)):
            t.copy_(n)
        for t in (y, dx, y8):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for e in range(G):
            a, b = int(off[e]), int(off[e + 1])
            assert torch.equal(y[a:b], (x[a:b].double() @ w[e].double().T).to(BF))
            assert torch.equal(dx[a:b], (dy[a:b].double() @ w[e].double()).to(BF))
            assert torch.equal(dw[e], (dy[a:b].double().T @ x[a:b].double()).float())
            if b > a:
                assert torch.equal(y8[a:b], fp8_ref(xq[a:b], sx[a:b], wq[e], sw[e])[0].to(BF))
        assert (y[sum(counts):] == 7).all() and (y8[sum(counts):] == 7).all()


def test_on_another_stream(api):
    counts, N, H = [40, 300], 520, 264
    x, dy, w, off = ragged(counts, N, H, gen(21), 0, 0)
    handle = api.MoeGemmRagged(2, 340, N, H, DEV)
    want = handle.forward(x, w, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = handle.forward(x, w, off, stream=side)
    q, s = api.quantize_blocks_fp8(x[:, :256].contiguous(), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    check_quant(x[:, :256].contiguous(), 1, q, s)


def test_two_handles_on_two_streams(api):
    """Each takes every SM: one after another, whatever the streams say."""
    N, H = 520, 1032
    sets = []
    for i, counts in enumerate(([300, 2, 0, 90], [1, 1, 500, 60])):
        x, dy, w, off = ragged(counts, N, H, gen(30 + i), 0, 0)
        handle = api.MoeGemmRagged(4, sum(counts), N, H, DEV)
        sets.append((handle, x, dy, w, off, torch.cuda.Stream(), handle.forward(x, w, off),
                     handle.weight_grad(dy, x, off)))
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for handle, x, dy, w, off, st, y, dw in sets:
            with torch.cuda.stream(st):
                got.append((handle.forward(x, w, off), handle.weight_grad(dy, x, off)))
        torch.cuda.synchronize()
        for (y2, dw2), s in zip(got, sets):
            assert torch.equal(y2, s[6]) and torch.equal(dw2, s[7])


def test_refusals(api):
    handle = api.MoeGemmRagged(2, 8, 16, 24, DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    x, dy = ints((8, 24), 1, gen(0)), ints((8, 16), 1, gen(0))
    w = ints((2, 16, 24), 1, gen(0))
    for bad in (lambda: handle.forward(x.float(), w, off), lambda: handle.forward(x, w, off.long()),
                lambda: handle.forward(x, w, off[:2]), lambda: handle.forward(x, w[:1], off),
                lambda: handle.forward(x[:, :16], w, off), lambda: handle.forward(x.cpu(), w, off),
                lambda: handle.input_grad(x, w, off), lambda: handle.weight_grad(dy, x[:4], off),
                lambda: handle.weight_grad(dy, x, off, dtype=torch.float16),
                lambda: handle.weight_grad(dy, x, off, accumulate=True),
                lambda: handle.weight_grad(dy, x, off, out=torch.empty((2, 16, 24), dtype=BF,
                                                                       device=DEV), accumulate=True),
                lambda: handle.forward(x, w, off, out=dy[:4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(api.MoeA2AError) as e:
        handle.forward(ints((9, 24), 1, gen(0)), w, off)
    assert e.value.status == api.MOE_ERR_CAPACITY
    odd = api.MoeGemmRagged(2, 8, 12, 24, DEV)           # N = 12: forward alone
    w12, dy12 = ints((2, 12, 24), 1, gen(0)), ints((8, 12), 1, gen(0))
    odd.forward(x, w12, off)
    for bad in (lambda: odd.input_grad(dy12, w12, off), lambda: odd.weight_grad(dy12, x, off)):
        with pytest.raises(api.MoeA2AError):
            bad()
    eight = api.MoeGemmFp8(2, 8, 16, 32, DEV)
    xq, sx, wq, sw = fp8_inputs((2,), 2, 8, 16, 32, gen(0))
    cnt = torch.zeros(2, dtype=torch.int32, device=DEV)
    for bad in (lambda: eight.gemm(xq.float(), sx, wq, sw), lambda: eight.gemm(xq, sx[..., 0], wq, sw),
                lambda: eight.gemm(xq, sx, wq, sw[:1]), lambda: eight.gemm(xq[0], sx[0], wq, sw),
                lambda: eight.gemm(xq, sx, wq, sw, counts=cnt.long()),
                lambda: eight.gemm(xq, sx, wq, sw, offsets=off),
                lambda: eight.gemm(xq[0], sx[0], wq, sw, counts=cnt, offsets=off)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: api.quantize_blocks_fp8(x, 2), lambda: api.quantize_blocks_fp8(x[0], 128),
                lambda: api.quantize_blocks_fp8(x.half()), lambda: api.quantize_blocks_fp8(x.cpu()),
                lambda: api.quantize_blocks_fp8(x, counts=cnt),
                lambda: api.quantize_blocks_fp8(torch.zeros((2, 4, 32), device=DEV), 128, counts=cnt)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(api.MoeA2AError):
        api.quantize_blocks_fp8(x)                       # 24 is no multiple of 16
