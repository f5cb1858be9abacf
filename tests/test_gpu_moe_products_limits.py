"""The experts' products at the ends of what their entry points take: offsets that
descend, very long sums, tensors that require gradients."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"
BF, F8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32


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


def offsets(values):
    return torch.tensor(values, dtype=I32, device=DEV)


def untouched(t, value):
    return all((part == value).all() for part in t.split(1 << 20))


# (tests/test_moe_tiling.py goes through the counts of these offsets)
def test_descending_offsets_whose_tiles_wrap_to_a_few(api):
    G, M, N, H = 1024, (1 << 28) + 1, 8, 8
    off = offsets([0] + [1 << 28, 0] * 500 + [M, 0] * 12)
    x = torch.ones((M, H), dtype=BF, device=DEV)
    out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    w = torch.ones((G, N, H), dtype=BF, device=DEV)
    handle = api.MoeGemmRagged(G, M, N, H, DEV)
    handle.forward(x, w, off, out=out)
    assert untouched(out, 7)
    handle.input_grad(x, w, off, out=out)
    assert untouched(out, 7)
    handle.forward(x, w, off.sort()[0], out=out)         # the call after it works
    assert untouched(out, 8)
    assert handle.get_error() == (api.MOE_OK, 0)


def test_descending_offsets_of_the_narrow_eight_bit_product(api):
    G, M, N, H = 1024, 48000, 180000, 16
    off = offsets([M if g % 2 else 0 for g in range(G + 1)])
    xq = torch.ones((M, H), device=DEV).to(F8)
    sx = torch.ones((M, 1), device=DEV)
    wq = torch.ones((1, 1, 1), device=DEV).to(F8).view(torch.uint8).expand(G, N, H).contiguous()
    sw = torch.ones((G, (N + 127) // 128, 1), device=DEV)
    out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    handle = api.MoeGemmFp8(G, M, N, H, DEV)
    handle.gemm(xq, sx, wq, sw, offsets=off, out=out)
    assert all((part == 7).all() for part in out.split(4000))
    few = torch.zeros_like(off)
    few[1:] = 40                                         # ascending ones
    handle.gemm(xq, sx, wq, sw, offsets=few, out=out)
    assert (out[:40] == 16).all() and (out[40:4000] == 7).all()
    assert handle.get_error() == (api.MOE_OK, 0)


@pytest.mark.parametrize("G,big,each", [(40, (1 << 29) + 17, 3), (400, (1 << 29) + 17, 3),
                                        (400, 1 << 29, 64)])
def test_weight_grad_of_a_tile_that_takes_seconds(api, G, big, each):
    """All rows but a few in one group, whose tile is not cut (40 tiles), or has others
    behind it (400), with and without a last block that is not full: the waits for it go
    past their usual limit."""
    N, H = 8, 8
    counts = [each] * G
    counts[3] = big
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    M = off[-1]
    g = gen(G)
    # most rows hold zeros, so the sums are exact
    x, dy = torch.zeros((M, H), dtype=BF, device=DEV), torch.zeros((M, N), dtype=BF, device=DEV)
    at = torch.randint(M, (2000,), generator=g, device=DEV)
    at = torch.cat([at, torch.arange(3 * G, device=DEV), M - 1 - torch.arange(3 * G, device=DEV)])
    for t in (x, dy):
        t[at] = torch.randint(-2, 3, (len(at), 8), generator=g, device=DEV).to(BF)
    handle = api.MoeGemmRagged(G, M, N, H, DEV)
    dw = handle.weight_grad(dy, x, offsets(off), dtype=F32)
    assert handle.get_error() == (api.MOE_OK, 0)
    live = at.unique()
    for e in range(G):
        rows = live[(live >= off[e]) & (live < off[e + 1])]
        assert torch.equal(dw[e].double(), dy[rows].double().T @ x[rows].double())


def one_sided(shape, g):
    return torch.rand(shape, generator=g, device=DEV) + 0.5


@pytest.mark.parametrize("way", ["forward", "input_grad"])
def test_long_sums_of_one_sign_are_not_biased(api, way):
    """As many tiles as pairs of 256 x 256 tiles' CTAs, so that none is cut along k.

    Truncating additions lose at most 2^-23 of the sum so far each: over 8192 terms that
    grow it evenly, 8192 * 2^-23 / 2 = 4.9e-4 of it.  (Without an end, 2^18 terms lost
    1.6e-3.)  The sums of those to nearest are 32 roundings of 2^-24.  The rounding to bf16,
    of outputs spread over a factor of four, is up or down by 2^-8 at most; the mean of n
    such is below 6 * 2^-8 / sqrt(3 n)."""
    k, lanes, M = (1 << 18) + 8, 76 * 256, 16
    g = gen(k)
    x = one_sided((M, k), g).to(BF)
    scale = 1 + torch.rand(lanes, generator=g, device=DEV)
    shape = (1, lanes, k) if way == "forward" else (1, k, lanes)
    w = torch.empty(shape, dtype=BF, device=DEV)
    maps = w[0] if way == "forward" else w[0].T          # [lanes, k]
    want = torch.empty((M, lanes), dtype=torch.float64, device=DEV)
    for i in range(0, lanes, 256):
        part = (one_sided((256, k), g) * scale[i:i + 256, None]).to(BF)
        maps[i:i + 256] = part
        want[:, i:i + 256] = x.double() @ part.double().T
    handle = api.MoeGemmRagged(1, M, lanes if way == "forward" else k,
                               k if way == "forward" else lanes, DEV)
    got = getattr(handle, way)(x, w, offsets([0, M])).double()
    assert handle.get_error() == (api.MOE_OK, 0)
    off = (got - want) / want
    lost = 8192 * 2.0 ** -23 / 2 + 32 * 2.0 ** -24
    assert off.abs().max() <= lost + 2.0 ** -8
    assert abs(off.mean()) <= lost + 6 * 2.0 ** -8 / (3 * off.numel()) ** 0.5


@pytest.mark.parametrize("lanes", [40, 256, 1000])
@pytest.mark.parametrize("k", [8192, 8200, 16384, 1 << 20])
def test_long_sums_of_integers(api, k, lanes):
    """Exact in fp32 (below 2^24), with parts that leave tensor memory once and more often."""
    off = offsets([0, 5, 5, 305])
    g = gen(k + lanes)
    three = lambda *s: torch.randint(-1, 2, s, generator=g, device=DEV, dtype=torch.int8).to(BF)
    x, w = three(305, k), three(3, lanes, k)
    up, down = (api.MoeGemmRagged(3, 305, n, h, DEV) for n, h in ((lanes, k), (k, lanes)))
    turned = w.transpose(1, 2).contiguous()              # [3, k, lanes]
    y, dx = up.forward(x, w, off), down.input_grad(x, turned, off)
    for e, (a, b) in enumerate(((0, 5), (5, 5), (5, 305))):
        want = (x[a:b].double() @ w[e].double().T).to(BF)
        assert torch.equal(y[a:b], want) and torch.equal(dx[a:b], want)
    assert up.get_error() == down.get_error() == (api.MOE_OK, 0)


def test_tensors_that_require_gradients(api):
    """forward refuses them where autograd expects a history, and works in a function of
    its own, whose gradients are the class's."""
    N, H = 24, 40
    off = offsets([0, 9, 9, 79])
    g = gen(2)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV).to(BF)
    x, w, dy = ints(79, H).requires_grad_(), ints(3, N, H).requires_grad_(), ints(79, N)
    handle = api.MoeGemmRagged(3, 79, N, H, DEV)

    class Map(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x, w)
            return handle.forward(x, w, off)

        @staticmethod
        def backward(ctx, dy):
            x, w = ctx.saved_tensors
            return handle.input_grad(dy, w, off), handle.weight_grad(dy, x, off)

    for tensors in ((x, w.detach()), (x.detach(), w)):
        with pytest.raises(ValueError, match="no history"):
            handle.forward(*tensors, off)
    with torch.no_grad():
        y = handle.forward(x, w, off)
    z = Map.apply(x, w)
    z.backward(dy)
    assert torch.equal(y, z) and z.requires_grad and not y.requires_grad
    a, b, d = x.detach().double(), w.detach().double(), dy.double()
    for e, (i, j) in enumerate(((0, 9), (9, 9), (9, 79))):
        assert torch.equal(y[i:j], (a[i:j] @ b[e].T).to(BF))
        assert torch.equal(x.grad[i:j], (d[i:j] @ b[e]).to(BF))
        assert torch.equal(w.grad[e], (d[i:j].T @ a[i:j]).to(BF))
    assert handle.get_error() == (api.MOE_OK, 0)


def test_fp32_weight_gradient_of_many_rows(api):
    """40 tiles, none of them cut, over 32768 rows of normal values.

    A run of 512 rows is 32 additions of the tensor cores, each of which loses at most
    2^-23 of what is there, which has grown with the root of their number: 2/3 * 32 * 2^-23
    = 2.6e-6 of the run's norm.  The 64 runs are added to nearest, at most 2^-24 each time:
    2/3 * 64 * 2^-24 = 2.6e-6.  Both are below 2^-17 = 7.6e-6; sums that stay in the tensor
    cores for all rows lose 1.1e-9 a row, 3.6e-5."""
    rows, N, H = 32768, 2048, 1280
    g = gen(5)
    x = torch.randn((rows, H), generator=g, device=DEV).to(BF)
    dy = torch.randn((rows, N), generator=g, device=DEV).to(BF)
    handle = api.MoeGemmRagged(1, rows, N, H, DEV)
    dw = handle.weight_grad(dy, x, offsets([0, rows]), dtype=F32)[0].double()
    want = dy.double().T @ x.double()
    assert (dw - want).norm() <= 2.0 ** -17 * want.norm()
    assert handle.get_error() == (api.MOE_OK, 0)
