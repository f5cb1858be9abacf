"""Sums that go through global memory, many times over: tiles cut by k between CTAs
and the layer's exchanges of activations and outputs.  Every call has other values,
so a part read too early is a wrong one.

The 8-bit product's sums are exact integers below 2^24.  The layer's weights pick
single values (one entry a row, powers of two), so its products are exact too.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"


@pytest.fixture(scope="module")
def api():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("M,N,H", [(16, 7168, 4096), (300, 1100, 7168), (5, 500, 16384)])
def test_product_of_cut_tiles_call_after_call(api, M, N, H):
    g = gen(M)
    h = api.MoeGemmInt8(1, M, N, H, DEV)
    ones = [torch.ones((1, n), device=DEV) for n in (M, N)]
    for _ in range(60):
        xq = torch.randint(-30, 31, (1, M, H), generator=g, device=DEV).to(torch.int8)
        wq = torch.randint(-30, 31, (1, N, H), generator=g, device=DEV).to(torch.int8)
        out = [h.gemm(xq, ones[0], wq, ones[1]) for _ in range(3)]
        # (|sums| <= 900 * 16384 < 2^24: fp32 holds them)
        ref = (xq[0].double() @ wq[0].double().T).to(torch.float32).to(torch.bfloat16)
        for o in out:
            assert torch.equal(o[0].view(torch.int16), ref.view(torch.int16))
    assert h.get_error() == (0, 0)


@pytest.mark.parametrize("T,E,H,I,K", [(1, 16, 2048, 768, 8), (8, 3, 2048, 4096, 2),
                                       (33, 2, 7168, 512, 1)])
def test_layer_of_cut_tiles_call_after_call(api, T, E, H, I, K):
    g = gen(T)
    h = api.MoeLayerSmall(E, H, I, K, T, api.MOE_FORMAT_BF16, DEV)
    for turn in range(40):
        # gate rows pick 16 x[c] (silu(z) is z in fp32 for z past 18), up rows
        # x[d]; W2 rows pick one activation
        c, d = (torch.randint(0, H, (E, I), generator=g, device=DEV) for _ in range(2))
        j = torch.randint(0, I, (E, H), generator=g, device=DEV)
        w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
        w13[:, :I].scatter_(2, c[:, :, None], 16.0)
        w13[:, I:].scatter_(2, d[:, :, None], 1.0)
        w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device=DEV)
        w2.scatter_(2, j[:, :, None], 1.0)
        x = torch.randint(2, 9, (T, H), generator=g, device=DEV).to(torch.bfloat16)
        ids = torch.topk(torch.rand((T, E), generator=g, device=DEV), K, dim=-1).indices
        w = torch.exp2(-torch.randint(0, 3, (T, K), generator=g, device=DEV).float())
        ref = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        X = x.double()
        for t in range(T):
            for k in range(K):
                e = int(ids[t, k])
                a = 16 * X[t, c[e]] * X[t, d[e]]
                ref[t] += float(w[t, k]) * a[j[e]]
        out = [h.forward(x, ids.int().contiguous(), w, w13, w2) for _ in range(3)]
        for o in out:                                   # (exact up to the narrowing to bf16)
            assert torch.equal(o.view(torch.int16), ref.to(torch.bfloat16).view(torch.int16)), turn
    assert h.get_error() == (0, 0)
