"""The experts' products and the block quantiser as they are used together: a
training step around the router's gate, an 8-bit expert behind a dispatch, and sizes
whose offsets pass 32 bits.

Integers and powers of two keep every fp32 sum exact (below 2^24), so outputs equal the
64-bit ones rounded where the operators round.
"""
import numpy as np
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


def ints(shape, most, g):
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(BF)


def bf(x):
    return x.to(BF).double()


class Step:
    """One training step of a layer: experts of the gate, rows sorted by expert, two maps
    with a rectifier between them, the tokens' sums, and the way back."""

    def __init__(self, api, T, K, E, H, F):
        self.api, self.T, self.K, self.E, self.H, self.F = api, T, K, E, H, F
        self.up = api.MoeGemmRagged(E, T * K, F, H, DEV)
        self.down = api.MoeGemmRagged(E, T * K, H, F, DEV)
        self.dw1 = torch.zeros((E, F, H), dtype=F32, device=DEV)

    def run(self, logits, x, w1, w2, dout):
        ids, _ = self.api.topk_gate(logits, self.K)
        flat = ids.flatten().long()
        order = torch.argsort(flat, stable=True)
        token = order // self.K
        first = torch.searchsorted(flat[order].contiguous(),
                                   torch.arange(self.E + 1, device=DEV)).to(I32)
        xs = x[token]
        y1 = self.up.forward(xs, w1, first)
        a = torch.relu(y1)
        y2 = self.down.forward(a, w2, first)
        out = torch.zeros((self.T, self.H), device=DEV).index_add_(0, token, y2.float())
        dy2 = dout[token]
        da = self.down.input_grad(dy2, w2, first)
        dw2 = self.down.weight_grad(dy2, a, first, dtype=F32)
        dy1 = torch.where(y1 > 0, da, torch.zeros_like(da))
        dxs = self.up.input_grad(dy1, w1, first)
        self.up.weight_grad(dy1, xs, first, out=self.dw1, accumulate=True)
        dx = torch.zeros((self.T, self.H), device=DEV).index_add_(0, token, dxs.float())
        return ids, out, dx, dw2

    def inputs(self, seed):
        g = gen(seed)
        logits = torch.randn((self.T, self.E), generator=g, device=DEV)
        logits[:, 0] += 1.5                              # uneven
        logits[:, self.E - 1] = -9.0                     # an expert without rows
        return [logits, ints((self.T, self.H), 2, g), ints((self.E, self.F, self.H), 1, g),
                ints((self.E, self.H, self.F), 1, g), ints((self.T, self.H), 1, g)]

    def check(self, ids, out, dx, dw2, dw1, logits, x, w1, w2, dout):
        assert torch.equal(ids.long().sort(1)[0], logits.topk(self.K, 1)[1].sort(1)[0])
        x, w1, w2, dout = x.double(), w1.double(), w2.double(), dout.double()
        o, dxr = torch.zeros_like(x), torch.zeros_like(x)
        for e in range(self.E):
            t = (ids == e).any(1).nonzero()[:, 0]
            y1 = bf(x[t] @ w1[e].T)
            a = y1.clamp(min=0)
            o[t] += bf(a @ w2[e].T)
            dy1 = bf(dout[t] @ w2[e]) * (y1 > 0)
            dxr[t] += bf(dy1 @ w1[e])
            assert torch.equal(dw2[e].double(), dout[t].T @ a)
            assert torch.equal(dw1[e].double(), dy1.T @ x[t])
        assert torch.equal(out.double(), o) and torch.equal(dx.double(), dxr)


@pytest.mark.parametrize("T,K,E,H,F", [(1, 2, 4, 64, 72), (90, 3, 6, 136, 104),
                                       (1000, 4, 16, 256, 384)])
def test_training_step(api, T, K, E, H, F):
    step = Step(api, T, K, E, H, F)
    given = step.inputs(T)
    ids, out, dx, dw2 = step.run(*given)
    step.check(ids, out, dx, dw2, step.dw1, *given)
    assert step.up.get_error() == step.down.get_error() == (api.MOE_OK, 0)


def test_training_step_captured_and_replayed(api):
    """One graph, replayed with other tokens; eager calls between replays share the scratch."""
    step = Step(api, 200, 2, 8, 128, 136)
    given = step.inputs(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run(*given)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step.run(*given)
    for seed in (2, 3, 1):
        fresh = step.inputs(seed)
        for to, new in zip(given, fresh):
            to.copy_(new)
        step.dw1.zero_()
        graph.replay()
        step.check(*got, step.dw1, *fresh)
        step.dw1.zero_()
        step.check(*step.run(*fresh), step.dw1, *fresh)


def test_eight_bit_experts_behind_a_dispatch(api):
    """Expert-layout planes, quantised up to their counts, times block-scaled weights into
    the combine payload."""
    R, T, H, E, K = 2, 60, 256, 4, 2
    g = gen(7)
    ids = torch.rand((R, T, E), generator=g, device=DEV).topk(K, 2)[1].to(I32)
    w = torch.full((R, T, K), 0.5, device=DEV)
    x = ints((R, T, H), 4, g)
    x[:, :, ::128] = 7.0                                 # the largest of every block: scale 2^-6
    wf = ints((E, H, H), 4, g)
    wf[:, ::128, ::128] = 7.0
    a2a = api.MoeA2A(R, T, H, E, K, DEV, layout=api.MOE_LAYOUT_EXPERT)
    wq, sw = api.quantize_blocks_fp8(wf, 128)
    for _ in range(2):
        view = a2a.dispatch(ids, w, x)
        cap, counts = view.plane_stride, view.recv_counts
        handle = api.MoeGemmFp8(E, cap, H, H, DEV)
        xq, sx = api.quantize_blocks_fp8(view.recv_x, counts=counts)
        handle.gemm(xq, sx, wq, sw, counts=counts, out=a2a.combine_payload())
        out = a2a.combine(None, True)
        assert handle.get_error() == (api.MOE_OK, 0) and a2a.get_error() == (api.MOE_OK, 0)
        for e in range(E):
            c = int(counts[e])
            assert (sx[e, :c] == 2.0 ** -6).all() and (sw[e] == 2.0 ** -6).all()
        # 64 x and 64 w are codes exactly where |x|, |w| <= 4 and 7 (448): the products are exact
        want = torch.zeros((R, T, H), dtype=torch.float64, device=DEV)
        for e in range(E):
            for k in range(K):
                m = ids[..., k] == e
                want[m] += 0.5 * bf(x[m].double() @ wf[e].double().T)
        assert torch.equal(out.double(), bf(want))


@pytest.mark.parametrize("M", [33, 64, 65, 81, 100, 128])
def test_cut_tiles_of_planes_of_up_to_a_tile_of_rows(api, M):
    """Tiles of 256 channels, cut along a long hidden size."""
    G, N, H = 10, 2560, 8192
    g = gen(M)
    xq, wq = ints((G, M, H), 4, g).to(F8), ints((G, N, H), 4, g).to(F8)
    two = lambda *s: torch.exp2(torch.randint(-2, 3, s, generator=g, device=DEV).float())
    sx, sw = two(G, M, H // 128), two(G, N // 128, H // 128)
    handle = api.MoeGemmFp8(G, M, N, H, DEV)
    outs = [handle.gemm(xq, sx, wq, sw) for _ in range(3)]
    for e in range(G):
        x = xq[e].double() * sx[e].double().repeat_interleave(128, 1)
        w = wq[e].double() * sw[e].double().repeat_interleave(128, 1).repeat_interleave(128, 0)
        want = (x @ w.T).to(BF)
        assert all(torch.equal(out[e], want) for out in outs)
    assert handle.get_error() == (api.MOE_OK, 0)


def test_rows_whose_offsets_pass_32_bits(api):
    M, N, H, last = (1 << 27) + 5, 24, 32, 1000
    g = gen(3)
    # rows of the last group hold values, the others ones
    x = torch.ones((M, H), dtype=BF, device=DEV)
    x[-last:] = ints((last, H), 3, g)
    off = torch.tensor([0, 7, M - last, M], dtype=I32, device=DEV)
    w = ints((3, N, H), 2, g)
    handle = api.MoeGemmRagged(3, M, N, H, DEV)
    y = handle.forward(x, w, off)
    bounds = ((0, 7, 0), (7, 2000, 1), (M - last - 2000, M - last, 1), (M - last, M, 2))
    for a, b, e in bounds:
        assert torch.equal(y[a:b].double(), bf(x[a:b].double() @ w[e].double().T))
    dx = handle.input_grad(y, w, off)
    for a, b, e in bounds:
        assert torch.equal(dx[a:b].double(), bf(y[a:b].double() @ w[e].double()))
    del dx
    y[7:M - last] = 0.0
    dw = handle.weight_grad(y, x, off, dtype=F32)
    for a, b, e in ((0, 7, 0), (M - last, M, 2)):
        assert torch.equal(dw[e].double(), y[a:b].double().T @ x[a:b].double())
    assert not dw[1].any()
    del y
    assert handle.get_error() == (api.MOE_OK, 0)
    # 8 bits: codes 64 x and 64 w of scales 2^-6
    x[:, 0], w[:, 0, 0] = 7.0, 7.0
    xq, sx = api.quantize_blocks_fp8(x)
    wq, sw = api.quantize_blocks_fp8(w, 128)
    eight = api.MoeGemmFp8(3, M, N, H, DEV)
    y = eight.gemm(xq, sx, wq, sw, offsets=off)
    for a, b, e in bounds:
        assert torch.equal(y[a:b].double(), bf(x[a:b].double() @ w[e].double().T))
    assert eight.get_error() == (api.MOE_OK, 0)


def test_descending_offsets_that_count_too_many_tiles(api):
    """Offsets that give all rows to every other group, at a size where the tiles would not
    be counted in 32 bits: no work, and no error."""
    G, M, N, H = 1024, 1 << 27, 1, 8
    x = torch.ones((M, H), dtype=BF, device=DEV)
    w = torch.ones((G, N, H), dtype=BF, device=DEV)
    off = torch.zeros(G + 1, dtype=I32, device=DEV)
    off[1::2] = M
    out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    handle = api.MoeGemmRagged(G, M, N, H, DEV)
    handle.forward(x, w, off, out=out)
    assert (out == 7).all()
    off[1:] = M                                          # and ascending ones, all in group 0
    handle.forward(x, w, off, out=out)
    assert (out == 8).all()
    assert handle.get_error() == (api.MOE_OK, 0)


@pytest.mark.parametrize("counts", [[512] * 6, [0, 1, 700, 64, 0, 1300], [40] * 80])
@pytest.mark.parametrize("N,H", [(264, 384), (1000, 1024), (520, 200)])
def test_weight_grad_added_to_what_is_there(api, counts, N, H):
    """Whole and cut tiles, with and without boxes; an expert without rows keeps every bit."""
    G, rows = len(counts), sum(counts)
    g = gen(N)
    x, dy = ints((rows, H), 2, g), ints((rows, N), 2, g)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=I32, device=DEV)
    handle = api.MoeGemmRagged(G, rows, N, H, DEV)
    start = torch.randint(-1000, 1000, (G, N, H), generator=g, device=DEV).float()
    start[torch.tensor(counts, device=DEV) == 0] = float("nan")
    dw = start.clone()
    for _ in range(3):
        handle.weight_grad(dy, x, off, out=dw, accumulate=True)
    o = off.tolist()
    for e in range(G):
        if counts[e] == 0:
            assert torch.equal(dw[e].view(I32), start[e].view(I32))
            continue
        one = dy[o[e]:o[e + 1]].double().T @ x[o[e]:o[e + 1]].double()
        assert torch.equal(dw[e].double(), start[e].double() + 3 * one)
    # normal values: one more rounding, of the sum, to the nearest
    real = torch.randn((rows, H), generator=g, device=DEV).to(BF)
    fresh = handle.weight_grad(dy, real, off, dtype=F32)
    base = torch.randn((G, N, H), generator=g, device=DEV)
    dw = base.clone()
    handle.weight_grad(dy, real, off, out=dw, accumulate=True)
    assert torch.equal(dw, base + fresh)
    assert handle.get_error() == (api.MOE_OK, 0)


@pytest.mark.parametrize("H", [128, 136])
def test_sums_below_the_smallest_normal_number_are_added(api, H):
    """2^-140 as a product, added to 2^-140 and to nothing."""
    off = torch.tensor([0, 64], dtype=I32, device=DEV)
    x = torch.zeros((64, H), dtype=BF, device=DEV)
    dy = torch.zeros((64, 256), dtype=BF, device=DEV)
    x[0, :2] = dy[0, 0] = 2.0 ** -70
    dw = torch.zeros((1, 256, H), device=DEV)
    dw[0, 0, 1:3] = 2.0 ** -140
    api.MoeGemmRagged(1, 64, 256, H, DEV).weight_grad(dy, x, off, out=dw, accumulate=True)
    want = torch.zeros((1, 256, H), dtype=torch.float64)
    want[0, 0, :3] = torch.tensor([1.0, 2.0, 1.0], dtype=torch.float64) * 2.0 ** -140
    assert torch.equal(dw.double().cpu(), want)
